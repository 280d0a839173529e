// delta_join.cu -- the chunked gated delta rule in segments: the states before
// the segments from what each does to a state, S <- M S + N from the first to
// the last, and backward the state's gradients behind them, dS <- M^T dS + dN
// from the last to the first.
//
// A block has 16 columns of one sequence's and head's state in shared memory, a
// thread one row of the result and 8 of the columns; M (by columns going
// forward, by rows going back: the row index runs over the threads) comes into
// shared memory one segment ahead. Read from L2 in the loop instead a segment
// took 11 us. Measured: 8 heads of 128 x 128 in 18 segments 37 us.
#include "delta.cuh"
#include "s4dplr.h"

namespace s4 {
namespace {

using namespace delta;

constexpr int kJoinCols = 16;

template <bool BACK>
__global__ void __launch_bounds__(256) k_delta_join(DeltaArgs a, const float *init, float *sums, bool keep,
                                                    unsigned *flags) {
    extern __shared__ __align__(128) float Ms[];   // [2][dk][dk]
    __shared__ float S[128][kJoinCols];
    __shared__ uint64_t full[2];
    const Summaries su(a.dk, a.dv, keep);
    const int hv = blockIdx.x % a.hv, s = blockIdx.x / a.hv, v0 = blockIdx.y * kJoinCols;
    const int d = threadIdx.x & 127, c0 = (threadIdx.x >> 7) * 8, mm = a.dk * a.dk;
    const int all = (sequence(a, s).len + kC - 1) / kC;
    const int n = all > a.seg ? (all + a.seg - 1) / a.seg : 1;
    const long long first = segment0(a, s);
    const bool in = d < a.dk && v0 + c0 < a.dv;   // dv is a multiple of 8
    auto unit = [&](int g) { return (size_t)((first + (BACK ? n - 1 - g : g)) * a.hv + hv); };
    auto fetch = [&](int g) {   // by one thread
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
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        x[j] = in && init ? __ldg(init + (((size_t)s * a.hv + hv) * a.dk + d) * a.dv + v0 + c0 + j) : 0.0f;
    bool ok = true;
    for (int g = 0;; ++g) {
        const size_t at = (size_t)d * a.dv + v0 + c0;
        if (in) {
            float4 *to = reinterpret_cast<float4 *>((BACK ? su.behind(sums, unit(g)) : su.start(sums, unit(g))) + at);
            to[0] = make_float4(x[0], x[1], x[2], x[3]);
            to[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
        if (g + 1 >= n) break;
        float4 p, q;
        if (in) {
            const float4 *np = reinterpret_cast<const float4 *>((BACK ? su.dn(sums, unit(g)) : su.n(sums, unit(g))) + at);
            p = np[0];
            q = np[1];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) S[d][c0 + j] = x[j];
        __syncthreads();   // S is there; the other half of Ms is used up
        if (threadIdx.x == 0 && g + 2 < n) fetch(g + 1);
        ok = umma::mbar_wait(full + (g & 1), (g >> 1) & 1, kSpinLimit) && ok;
        if (in) {
            x[0] = p.x, x[1] = p.y, x[2] = p.z, x[3] = p.w, x[4] = q.x, x[5] = q.y, x[6] = q.z, x[7] = q.w;
            const float *M = Ms + (g & 1) * mm + d;
            const int columns = BACK || g > 0 || init ? a.dk : 0;   // the first M is not there for a state of zeros
#pragma unroll 8
            for (int c = 0; c < columns; ++c) {
                const float m = M[c * a.dk];
                const float4 u = *reinterpret_cast<const float4 *>(&S[c][c0]);
                const float4 w = *reinterpret_cast<const float4 *>(&S[c][c0 + 4]);
                x[0] = fmaf(m, u.x, x[0]);
                x[1] = fmaf(m, u.y, x[1]);
                x[2] = fmaf(m, u.z, x[2]);
                x[3] = fmaf(m, u.w, x[3]);
                x[4] = fmaf(m, w.x, x[4]);
                x[5] = fmaf(m, w.y, x[5]);
                x[6] = fmaf(m, w.z, x[6]);
                x[7] = fmaf(m, w.w, x[7]);
            }
        }
        __syncthreads();
    }
    if (!ok && flags && threadIdx.x == 0) atomicOr(flags, S4_FLAG_TIMEOUT);
}

template <bool BACK>
cudaError_t run(const DeltaArgs &a, const float *init, float *sums, bool keep, unsigned *flags, cudaStream_t st) {
    static SmemLimit limit;
    cudaError_t e = limit.raise(k_delta_join<BACK>, 2 * 128 * 128 * sizeof(float));
    if (e != cudaSuccess) return e;
    k_delta_join<BACK><<<dim3(a.n * a.hv, (a.dv + kJoinCols - 1) / kJoinCols), 256, 2 * a.dk * a.dk * sizeof(float), st>>>(
        a, init, sums, keep, flags);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_join(const DeltaArgs &a, const float *init, float *sums, bool keep, bool back, unsigned *flags,
                              cudaStream_t st) {
    return back ? run<true>(a, init, sums, keep, flags, st) : run<false>(a, init, sums, keep, flags, st);
}

}  // namespace s4
