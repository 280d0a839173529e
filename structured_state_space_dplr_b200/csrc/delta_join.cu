// delta_join.cu -- the chunked gated delta rule in segments: the states before
// the segments from what each does to a state, S <- M S + N from the first to
// the last, and backward the state's gradients behind them, dS <- M^T dS + dN
// from the last to the first.
//
// A block has 16 columns of one sequence's and head's state in shared memory, a
// thread 4 rows and 4 columns of the result: two 16-byte reads for 16 products
// (one row and 8 columns a thread: 77 us for what takes 49, most of it reads of
// S), those of 8 products read before them (left to the compiler 53 to 82 us,
// with the code around the loop). M (by columns going forward, by rows going
// back: the row index runs over the threads) comes into shared memory one segment
// ahead. Bound by the segments one after the other. Measured: 65536 tokens, 8
// heads of 128 x 128 49 us.
#include "delta.cuh"
#include "s4dplr.h"

namespace s4 {
namespace {

using namespace delta;

constexpr int kJoinCols = 16, kJoinThreads = 128;

__device__ __forceinline__ float4 fma4(float a, float4 b, float4 c) {
    return make_float4(fmaf(a, b.x, c.x), fmaf(a, b.y, c.y), fmaf(a, b.z, c.z), fmaf(a, b.w, c.w));
}

template <bool BACK>
__global__ void __launch_bounds__(kJoinThreads) k_delta_join(DeltaArgs a, const float *init, float *sums, bool keep,
                                                    unsigned *flags) {
    extern __shared__ __align__(128) float Ms[];   // [2][dk][dk]
    __shared__ __align__(16) float S[128][kJoinCols];
    __shared__ uint64_t full[2];
    const Summaries su(a.dk, a.dv, keep);
    const int hv = blockIdx.x % a.hv, s = blockIdx.x / a.hv, v0 = blockIdx.y * kJoinCols;
    const int r0 = (threadIdx.x >> 2) * 4, c0 = (threadIdx.x & 3) * 4, mm = a.dk * a.dk;
    const int all = (sequence(a, s).len + kC - 1) / kC;
    const int n = all > a.seg ? (all + a.seg - 1) / a.seg : 1;
    const long long first = segment0(a, s);
    const bool in = r0 < a.dk && v0 + c0 < a.dv;   // dk and dv are multiples of 8
    auto unit = [&](int g) { return (size_t)((first + (BACK ? n - 1 - g : g)) * a.hv + hv); };
    int fetched = 0;
    auto fetch = [&](int g) {   // by one thread
        ++fetched;
        umma::fence_proxy_async();
        mbar_expect(full + (g & 1), mm * 4);
        bulk_load(Ms + (g & 1) * mm, BACK ? su.m_rows(sums, unit(g)) : su.m(sums, unit(g)), mm * 4, full + (g & 1));
        mbar_arrive(full + (g & 1));
    };
    if (threadIdx.x == 0) {
        umma::mbar_init(full, 1);
        umma::mbar_init(full + 1, 1);
        umma::fence_mbar_init();
        if (n > 1) fetch(0);
    }
    const size_t at = (size_t)r0 * a.dv + v0 + c0;
    auto rows4 = [&](const float *p, float4 (&f)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = *reinterpret_cast<const float4 *>(p + at + (size_t)j * a.dv);
    };
    float4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = make_float4(0, 0, 0, 0);
    if (in && init) rows4(init + ((size_t)s * a.hv + hv) * a.dk * a.dv, x);
    bool ok = true;
    for (int g = 0;; ++g) {
        if (in) {
            float *to = (BACK ? su.behind(sums, unit(g)) : su.start(sums, unit(g))) + at;
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<float4 *>(to + (size_t)j * a.dv) = x[j];
        }
        if (g + 1 >= n) break;
        float4 p[4];
        if (in) rows4(BACK ? su.dn(sums, unit(g)) : su.n(sums, unit(g)), p);   // on its way
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<float4 *>(&S[r0 + j][c0]) = x[j];
        __syncthreads();   // S is there; the other half of Ms is used up
        if (threadIdx.x == 0 && g + 2 < n) fetch(g + 1);
        ok = umma::mbar_wait(full + (g & 1), (g >> 1) & 1, kSpinLimit);
        if (in) {
            const float *M = Ms + (g & 1) * mm + r0;
            const int columns = BACK || g > 0 || init ? a.dk : 0;   // the first M is not there for a state of zeros
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = make_float4(0, 0, 0, 0);
            for (int c = 0; c < columns; c += 8) {   // dk is a multiple of 8
                float4 m[8], u[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    m[k] = *reinterpret_cast<const float4 *>(M + (c + k) * a.dk);
                    u[k] = *reinterpret_cast<const float4 *>(&S[c + k][c0]);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    x[0] = fma4(m[k].x, u[k], x[0]);
                    x[1] = fma4(m[k].y, u[k], x[1]);
                    x[2] = fma4(m[k].z, u[k], x[2]);
                    x[3] = fma4(m[k].w, u[k], x[3]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = fma4(1.0f, p[j], x[j]);
        }
        if (!__syncthreads_and(ok)) {
            ok = false;
            break;
        }
    }
    if (!ok && threadIdx.x == 0) drain_copies(full, fetched, 2);
    if (!ok && flags) atomicOr(flags, S4_FLAG_TIMEOUT);
}

template <bool BACK>
cudaError_t run(const DeltaArgs &a, const float *init, float *sums, bool keep, unsigned *flags, cudaStream_t st) {
    static SmemLimit limit;
    cudaError_t e = limit.raise(k_delta_join<BACK>, 2 * 128 * 128 * sizeof(float));
    if (e != cudaSuccess) return e;
    k_delta_join<BACK><<<dim3(a.n * a.hv, (a.dv + kJoinCols - 1) / kJoinCols), kJoinThreads, 2 * a.dk * a.dk * sizeof(float), st>>>(
        a, init, sums, keep, flags);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_join(const DeltaArgs &a, const float *init, float *sums, bool keep, bool back, unsigned *flags,
                              cudaStream_t st) {
    return back ? run<true>(a, init, sums, keep, flags, st) : run<false>(a, init, sums, keep, flags, st);
}

}  // namespace s4
