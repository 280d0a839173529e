// delta_scan.cu -- the gated delta rule token by token (decode): one or a few
// tokens per sequence, the state read and written once per call.
//
//     S <- a S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q
//
// The two products with the state are taken together before the update:
// o = scale (S^T q + (k.q) u) with the decayed S, so a token costs one pass
// over the state in registers and one barrier.
//
// Bound by memory: 8 Dk Dv bytes per head and call for the state, everything
// else is small. A block of 256 threads holds a [Dk, 4 LV] slice of one head's
// state, float4 columns across LV threads and the rows spread over the other
// 256 / LV, so all of the slice is in flight at once. LV = 32 covers Dv = 128
// in one block (64 KB in flight); with few heads in all, narrower slices give
// more blocks, and the latency of one block goes down with its rows per thread.
// Measured: 256 sequences of 32 heads of 128 x 128, 180 us for 1.08 GB (6.0
// TB/s, 92% of a plain copy's rate); one sequence of 16 heads 2.8 us.
#include "dtype.cuh"
#include "launch.h"
#include "s4dplr.h"

namespace s4 {
namespace {

constexpr int kMaxD = 128;

__device__ __forceinline__ float4 fma4(float a, float4 b, float4 c) {
    return make_float4(fmaf(a, b.x, c.x), fmaf(a, b.y, c.y), fmaf(a, b.z, c.z), fmaf(a, b.w, c.w));
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 shfl4(float4 a, int o) {
    return make_float4(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o),
                       __shfl_xor_sync(0xffffffffu, a.z, o), __shfl_xor_sync(0xffffffffu, a.w, o));
}

// q, k [Bt, T, Hk, Dk], v, o [Bt, T, Hv, Dv] (token strides sq, sk, sv in
// elements; o contiguous), g, beta [Bt, T, Hv], state [Bt, Hv, Dk, Dv]
template <typename T_, int LV>
__global__ void __launch_bounds__(256) k_delta_scan(const T_ *__restrict__ q, const T_ *__restrict__ k,
                                                    const T_ *__restrict__ v, const float *__restrict__ g,
                                                    const float *__restrict__ beta, float *state, int T, int Hk,
                                                    int Hv, int Dk, int Dv, long long sq, long long sk, long long sv,
                                                    float scale, T_ *o) {
    constexpr int RG = 256 / LV;          // row groups
    constexpr int R = kMaxD / RG;         // rows per thread
    __shared__ float sk_[2][kMaxD], sq_[2][kMaxD];
    __shared__ float4 red[2][8][2][LV];   // per warp: S^T k, S^T q
    const int tid = threadIdx.x, lv = tid % LV, rg = tid / LV, warp = tid >> 5;
    const int hv = blockIdx.x % Hv, b = blockIdx.x / Hv, hk = hv / (Hv / Hk);
    const int c = blockIdx.y * 4 * LV + 4 * lv;
    const bool in = c < Dv;               // Dv is a multiple of 8: c < Dv implies c + 3 < Dv
    float *sp = state + ((size_t)b * Hv + hv) * Dk * Dv + c;
    const long long tok0 = (long long)b * T;
    float4 S[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = rg + RG * i;
        S[i] = in && r < Dk ? *reinterpret_cast<const float4 *>(sp + (size_t)r * Dv) : make_float4(0, 0, 0, 0);
    }
    // the token's k and q: one element a thread
    auto fetch = [&](int t) {
        const int e = tid & 127;
        if (e >= Dk) return 0.0f;
        return tid < 128 ? to_f(k[(tok0 + t) * sk + (long long)hk * Dk + e])
                         : to_f(q[(tok0 + t) * sq + (long long)hk * Dk + e]);
    };
    float next = fetch(0);
    for (int t = 0; t < T; ++t) {
        const int p = t & 1;
        (tid < 128 ? sk_ : sq_)[p][tid & 127] = next;
        const long long tok = tok0 + t;
        const float a = expf(__ldg(g + tok * Hv + hv)), be = __ldg(beta + tok * Hv + hv);
        float vv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (in) load_pack<T_, 4>(v + tok * sv + (long long)hv * Dv + c, vv);
        if (t + 1 < T) next = fetch(t + 1);
        __syncthreads();
        float4 ak = make_float4(0, 0, 0, 0), aq = ak;
        float kr[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = rg + RG * i;
            kr[i] = sk_[p][r];            // rows past Dk hold zero
            S[i] = make_float4(S[i].x * a, S[i].y * a, S[i].z * a, S[i].w * a);
            ak = fma4(kr[i], S[i], ak);
            aq = fma4(sq_[p][r], S[i], aq);
        }
        float kq = 0.0f;                  // k.q, by every warp for itself
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i) kq = fmaf(sk_[p][(tid & 31) + 32 * i], sq_[p][(tid & 31) + 32 * i], kq);
#pragma unroll
        for (int s = 16; s; s >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, s);
#pragma unroll
        for (int s = LV; s < 32; s <<= 1) {
            ak = add4(ak, shfl4(ak, s));
            aq = add4(aq, shfl4(aq, s));
        }
        if ((tid & 31) < LV) {
            red[p][warp][0][lv] = ak;
            red[p][warp][1][lv] = aq;
        }
        __syncthreads();
        ak = red[p][0][0][lv];
        aq = red[p][0][1][lv];
#pragma unroll
        for (int w = 1; w < 8; ++w) {
            ak = add4(ak, red[p][w][0][lv]);
            aq = add4(aq, red[p][w][1][lv]);
        }
        const float4 u = make_float4(be * (vv[0] - ak.x), be * (vv[1] - ak.y), be * (vv[2] - ak.z), be * (vv[3] - ak.w));
#pragma unroll
        for (int i = 0; i < R; ++i) S[i] = fma4(kr[i], u, S[i]);
        if (rg == 0 && in) {
            const float ov[4] = {scale * fmaf(kq, u.x, aq.x), scale * fmaf(kq, u.y, aq.y),
                                 scale * fmaf(kq, u.z, aq.z), scale * fmaf(kq, u.w, aq.w)};
            store_pack<T_, 4>(o + (tok * Hv + hv) * Dv + c, ov);
        }
    }
    if (!in) return;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = rg + RG * i;
        if (r < Dk) *reinterpret_cast<float4 *>(sp + (size_t)r * Dv) = S[i];
    }
}

template <typename T_>
void run(int lv, const DeltaArgs &a, float *state, int T, cudaStream_t st) {
    dim3 grid((unsigned)(a.n * a.hv), (unsigned)((a.dv + 4 * lv - 1) / (4 * lv)));
    auto go = [&](auto f) {
        f<<<grid, 256, 0, st>>>((const T_ *)a.q, (const T_ *)a.k, (const T_ *)a.v, a.g, a.beta, state, T, a.hk, a.hv,
                                a.dk, a.dv, a.sq, a.sk, a.sv, a.scale, (T_ *)a.o);
    };
    if (lv == 32)
        go(k_delta_scan<T_, 32>);
    else if (lv == 16)
        go(k_delta_scan<T_, 16>);
    else
        go(k_delta_scan<T_, 8>);
}

}  // namespace

cudaError_t launch_delta_scan(int dtype, const DeltaArgs &a, float *state, int T, cudaStream_t st) {
    if (a.n == 0 || T == 0) return cudaSuccess;
    const long long heads = (long long)a.n * a.hv;
    const int lv = heads >= 2 * 148 ? (a.dv > 64 ? 32 : a.dv > 32 ? 16 : 8) : heads >= 148 && a.dv > 32 ? 16 : 8;
    if (dtype == S4_BF16)
        run<__nv_bfloat16>(lv, a, state, T, st);
    else if (dtype == S4_F16)
        run<__half>(lv, a, state, T, st);
    else
        run<float>(lv, a, state, T, st);
    return cudaGetLastError();
}

}  // namespace s4
