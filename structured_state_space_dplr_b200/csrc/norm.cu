// norm.cu -- layer norm over token rows (forward and backward) and the
// backward of the S4Block's norm over channels.
//
//   xhat = (x - mu) rstd,  z = xhat gamma + beta,  rstd = (var + eps)^-1/2
//   h = dz gamma,  dx = rstd (h - mean(h) - xhat mean(h xhat))
//   dgamma = sum over rows of dz xhat,  dbeta = sum over rows of dz
//
// Both directions move each array once (rows: forward x -> z, backward x, dz
// -> dx; channels: x, dz -> dx) and are bound by memory. A row is kept in
// registers between its reductions. The weight gradients are summed in
// registers over all rows a block visits (a fixed set, in a fixed order),
// written as one partial row per block and added up by a second small kernel
// in a fixed order: no atomics, the same bits every time.
#include "dtype.cuh"
#include "launch.h"
#include "s4dplr.h"

#include <type_traits>

namespace s4 {
namespace {

constexpr int kBlocks = 148 * 4;   // backward blocks: four per SM, each with a partial row of weight gradients

// Sum of N values over the group of `tpr` threads (a power of two) that holds
// a row. Groups of more than a warp go through shared memory: one barrier,
// two buffers in turn, so every thread of the block has to call it equally often.
template <int N, bool BIG>
__device__ __forceinline__ void group_sum(float (&v)[N], int tpr, float *buf, int &turn) {
    const int w = BIG ? 32 : tpr;
    for (int o = w >> 1; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (BIG) {
        float *b = buf + (turn & 1) * N * 32;
        ++turn;
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) b[i * 32 + warp] = v[i];
        __syncthreads();
        const int w0 = (threadIdx.x / tpr) * (tpr >> 5), nw = tpr >> 5;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.0f;
            for (int k = 0; k < nw; ++k) s += b[i * 32 + w0 + k];
            v[i] = s;
        }
    }
}

template <typename T, int V, int NV, bool BIG, int MAXT>
__global__ void __launch_bounds__(MAXT) k_layernorm_rows(const T *__restrict__ x,
                                                                     const float *__restrict__ gamma,
                                                                     const float *__restrict__ beta, float eps,
                                                                     long long rows, int D, int tpr, T *z,
                                                                     float *mean, float *rstd) {
    __shared__ float buf[2 * 32];
    int turn = 0;
    const int groups = blockDim.x / tpr, l = threadIdx.x % tpr;
    const long long row = (long long)blockIdx.x * groups + threadIdx.x / tpr;
    const bool in = row < rows;
    float v[NV][V];
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (l + i * tpr) * V;
        if (in && c < D) {
            load_pack<T, V>(x + row * D + c, v[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) s[0] += v[i][j];
        }
    }
    group_sum<1, BIG>(s, tpr, buf, turn);
    const float mu = s[0] / (float)D;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (in && (l + i * tpr) * V < D)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i][j] -= mu;
                s[0] = fmaf(v[i][j], v[i][j], s[0]);
            }
    group_sum<1, BIG>(s, tpr, buf, turn);
    const float rs = 1.0f / sqrtf(s[0] / (float)D + eps);
    if (!in) return;
    if (l == 0) {
        mean[row] = mu;
        rstd[row] = rs;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (l + i * tpr) * V;
        if (c < D) {
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = fmaf(v[i][j] * rs, __ldg(gamma + c + j), __ldg(beta + c + j));
            store_pack<T, V>(z + row * D + c, o);
        }
    }
}

template <typename T, int V, int NV, bool BIG, int MAXT>
__global__ void __launch_bounds__(MAXT) k_layernorm_rows_backward(
    const T *__restrict__ dz, const T *__restrict__ x, const float *__restrict__ gamma,
    const float *__restrict__ mean, const float *__restrict__ rstd, long long rows, int D, int tpr, T *dx,
    float *part) {
    __shared__ float buf[2 * 2 * 32];
    extern __shared__ float sacc[];   // groups > 1: [2][D]
    int turn = 0;
    const int groups = blockDim.x / tpr, l = threadIdx.x % tpr, gi = threadIdx.x / tpr;
    float dg[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) dg[i][j] = db[i][j] = 0.0f;
    const float inv = 1.0f / (float)D;
    const long long stride = (long long)gridDim.x * groups;
    // every group of a block takes the same number of turns (the barrier in group_sum)
    for (long long r0 = (long long)blockIdx.x * groups; r0 < rows; r0 += stride) {
        const long long row = r0 + gi;
        const bool in = row < rows;
        float xv[NV][V], h[NV][V];
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (l + i * tpr) * V;
            if (in && c < D) {
                load_pack<T, V>(x + row * D + c, xv[i]);
                load_pack<T, V>(dz + row * D + c, h[i]);
            }
        }
        const float mu = in ? __ldg(mean + row) : 0.0f, rs = in ? __ldg(rstd + row) : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in && (l + i * tpr) * V < D)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    xv[i][j] = (xv[i][j] - mu) * rs;
                    dg[i][j] = fmaf(h[i][j], xv[i][j], dg[i][j]);
                    db[i][j] += h[i][j];
                    h[i][j] *= __ldg(gamma + (l + i * tpr) * V + j);
                    s[0] += h[i][j];
                    s[1] = fmaf(h[i][j], xv[i][j], s[1]);
                }
        group_sum<2, BIG>(s, tpr, buf, turn);
        const float m0 = s[0] * inv, m1 = s[1] * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (l + i * tpr) * V;
            if (in && c < D) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = rs * (h[i][j] - fmaf(xv[i][j], m1, m0));
                store_pack<T, V>(dx + row * D + c, o);
            }
        }
    }
    float *p = part + (size_t)blockIdx.x * 2 * D;
    if (groups > 1) {   // the block's groups one after the other
        for (int g = 0; g < groups; ++g) {
            if (gi == g)
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const int c = (l + i * tpr) * V + j;
                        if (c < D) {
                            sacc[c] = (g ? sacc[c] : 0.0f) + dg[i][j];
                            sacc[D + c] = (g ? sacc[D + c] : 0.0f) + db[i][j];
                        }
                    }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * D; c += blockDim.x) p[c] = sacc[c];
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (l + i * tpr) * V + j;
                if (c < D) {
                    p[c] = dg[i][j];
                    p[D + c] = db[i][j];
                }
            }
    }
}

// out0[c], out1[c] = sums over n partial rows [2][D]: 32 columns a block, 8
// strided slices of the rows each, added in order
__global__ void __launch_bounds__(256) k_sum_partials(const float *__restrict__ part, int n, int D, float *out0,
                                                      float *out1) {
    __shared__ float s[8][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float a = 0.0f;
    if (c < 2 * D) {
        int r = w;
        for (; r + 24 < n; r += 32) {
            const float v0 = part[(size_t)r * 2 * D + c], v1 = part[(size_t)(r + 8) * 2 * D + c];
            const float v2 = part[(size_t)(r + 16) * 2 * D + c], v3 = part[(size_t)(r + 24) * 2 * D + c];
            a += (v0 + v1) + (v2 + v3);
        }
        for (; r < n; r += 8) a += part[(size_t)r * 2 * D + c];
    }
    s[w][threadIdx.x & 31] = a;
    __syncthreads();
    if (w == 0 && c < 2 * D) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += s[i][threadIdx.x];
        if (c < D)
            out0[c] = t;
        else
            out1[c - D] = t;
    }
}

// ---------------------------------------------------- channel layout ------
// x, dz [Bt, H, L]: a tile is 64 time steps of one batch row, 16 threads x 4
// steps wide and 16 slices of the channels deep.
constexpr int kSteps = 64, kSlices = 16;

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 sub4(float4 a, float4 b) {
    return make_float4(a.x - b.x, a.y - b.y, a.z - b.z, a.w - b.w);
}
__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
    return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float4 fma4(float4 a, float4 b, float4 c) {
    return make_float4(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y), fmaf(a.z, b.z, c.z), fmaf(a.w, b.w, c.w));
}
__device__ __forceinline__ float4 scale4(float4 a, float s) { return make_float4(a.x * s, a.y * s, a.z * s, a.w * s); }
__device__ __forceinline__ float sum4(float4 a) { return (a.x + a.y) + (a.z + a.w); }
__device__ __forceinline__ float4 rstd4(float4 ss, float inv, float eps) {
    return make_float4(1.0f / sqrtf(ss.x * inv + eps), 1.0f / sqrtf(ss.y * inv + eps),
                       1.0f / sqrtf(ss.z * inv + eps), 1.0f / sqrtf(ss.w * inv + eps));
}

// sum over the slices of a value per (slice, steps); two barriers
__device__ __forceinline__ float4 slice_sum(float4 a, float4 (*red)[kSteps / 4], int hs, int tl) {
    __syncthreads();
    red[hs][tl] = a;
    __syncthreads();
    float4 s = red[0][tl];
#pragma unroll
    for (int i = 1; i < kSlices; ++i) s = add4(s, red[i][tl]);
    return s;
}
// sum over the 16 threads of a slice
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// H <= 16 NV: x and dz of a tile stay in registers, and so do the weight
// gradients of the thread's channels over all tiles of the block
template <int NV>
__global__ void __launch_bounds__(256) k_layernorm_channels_backward_reg(
    const float *__restrict__ dz, const float *__restrict__ x, const float *__restrict__ gamma, float eps, int Bt,
    int H, int L, float *dx, float *part) {
    __shared__ float4 red[kSlices][kSteps / 4];
    const int tl = threadIdx.x % (kSteps / 4), hs = threadIdx.x / (kSteps / 4);
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float inv = 1.0f / (float)H;
    float dg[NV], db[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) dg[i] = db[i] = 0.0f;
    const int tiles_l = (L + kSteps - 1) / kSteps;
    const long long tiles = (long long)tiles_l * Bt;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int t = (int)(tile % tiles_l) * kSteps + 4 * tl;
        const bool in = t < L;   // L is a multiple of 16: t < L implies t + 3 < L
        const size_t base = (size_t)(tile / tiles_l) * H * L + t;
        float4 v[NV], w[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int h = hs + kSlices * i;
            const bool ok = in && h < H;
            v[i] = ok ? *reinterpret_cast<const float4 *>(x + base + (size_t)h * L) : zero;
            w[i] = ok ? *reinterpret_cast<const float4 *>(dz + base + (size_t)h * L) : zero;
        }
        float4 a = zero;
#pragma unroll
        for (int i = 0; i < NV; ++i) a = add4(a, v[i]);
        const float4 mu = scale4(slice_sum(a, red, hs, tl), inv);
        a = zero;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (hs + kSlices * i < H) {
                v[i] = sub4(v[i], mu);
                a = fma4(v[i], v[i], a);
            }
        const float4 rs = rstd4(slice_sum(a, red, hs, tl), inv, eps);
        float4 s0 = zero, s1 = zero;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int h = hs + kSlices * i;
            if (h < H) {
                v[i] = mul4(v[i], rs);
                dg[i] += sum4(mul4(w[i], v[i]));   // steps past L hold dz = 0
                db[i] += sum4(w[i]);
                w[i] = scale4(w[i], __ldg(gamma + h));
                s0 = add4(s0, w[i]);
                s1 = fma4(w[i], v[i], s1);
            }
        }
        const float4 m0 = scale4(slice_sum(s0, red, hs, tl), inv);
        const float4 m1 = scale4(slice_sum(s1, red, hs, tl), inv);
        if (in)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int h = hs + kSlices * i;
                if (h < H)
                    *reinterpret_cast<float4 *>(dx + base + (size_t)h * L) =
                        mul4(rs, sub4(w[i], fma4(v[i], m1, m0)));
            }
    }
    float *p = part + (size_t)blockIdx.x * 2 * H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int h = hs + kSlices * i;
        const float g = lane_sum(dg[i]), b = lane_sum(db[i]);
        if (h < H && tl == 0) {
            p[h] = g;
            p[H + h] = b;
        }
    }
}

// any H: the tile is read three times (mean; variance and the two sums of the
// gradient; output), the later reads mostly from L2, and the weight gradients
// are kept in shared memory, each channel's by the slice that owns it
__global__ void __launch_bounds__(256) k_layernorm_channels_backward(
    const float *__restrict__ dz, const float *__restrict__ x, const float *__restrict__ gamma, float eps, int Bt,
    int H, int L, float *dx, float *part) {
    __shared__ float4 red[kSlices][kSteps / 4];
    extern __shared__ float sacc[];   // [2][H]
    const int tl = threadIdx.x % (kSteps / 4), hs = threadIdx.x / (kSteps / 4);
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float inv = 1.0f / (float)H;
    for (int c = threadIdx.x; c < 2 * H; c += 256) sacc[c] = 0.0f;
    const int tiles_l = (L + kSteps - 1) / kSteps;
    const long long tiles = (long long)tiles_l * Bt;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int t = (int)(tile % tiles_l) * kSteps + 4 * tl;
        const bool in = t < L;
        const size_t base = (size_t)(tile / tiles_l) * H * L + t;
        float4 a = zero;
        if (in)
            for (int h = hs; h < H; h += kSlices)
                a = add4(a, *reinterpret_cast<const float4 *>(x + base + (size_t)h * L));
        const float4 mu = scale4(slice_sum(a, red, hs, tl), inv);
        float4 ss = zero, s0 = zero, s1 = zero;
        if (in)
            for (int h = hs; h < H; h += kSlices) {
                const float4 c = sub4(*reinterpret_cast<const float4 *>(x + base + (size_t)h * L), mu);
                const float4 w = scale4(*reinterpret_cast<const float4 *>(dz + base + (size_t)h * L), __ldg(gamma + h));
                ss = fma4(c, c, ss);
                s0 = add4(s0, w);
                s1 = fma4(w, c, s1);
            }
        const float4 rs = rstd4(slice_sum(ss, red, hs, tl), inv, eps);
        const float4 m0 = scale4(slice_sum(s0, red, hs, tl), inv);
        const float4 m1 = mul4(scale4(slice_sum(s1, red, hs, tl), inv), rs);
        const int hn = (H + kSlices - 1) / kSlices;
        for (int i = 0; i < hn; ++i) {   // the same count for all lanes: lane_sum is a warp operation
            const int h = hs + kSlices * i;
            float g = 0.0f, b = 0.0f;
            if (in && h < H) {
                const float4 xh = mul4(sub4(*reinterpret_cast<const float4 *>(x + base + (size_t)h * L), mu), rs);
                const float4 d = *reinterpret_cast<const float4 *>(dz + base + (size_t)h * L);
                g = sum4(mul4(d, xh));
                b = sum4(d);
                *reinterpret_cast<float4 *>(dx + base + (size_t)h * L) =
                    mul4(rs, sub4(scale4(d, __ldg(gamma + h)), fma4(xh, m1, m0)));
            }
            g = lane_sum(g);
            b = lane_sum(b);
            if (h < H && tl == 0) {
                sacc[h] += g;
                sacc[H + h] += b;
            }
        }
    }
    __syncthreads();
    float *p = part + (size_t)blockIdx.x * 2 * H;
    for (int c = threadIdx.x; c < 2 * H; c += 256) p[c] = sacc[c];
}

// How a row of D elements is spread: V per access, NV accesses by each of tpr
// threads, at most 16 elements a thread (8 when single): registers hold the
// row, its gradient and two weight gradients. D <= 8192 takes at most 512
// threads, or 1024 with single elements.
struct RowPlan { int v, nv, tpr, block; };

RowPlan row_plan(int D, int elem, bool vector) {
    RowPlan p;
    p.v = vector ? 16 / elem : 1;
    const int need = (D + p.v - 1) / p.v, most = vector ? 16 / p.v : 8;
    p.nv = 1;
    p.tpr = 1;
    while (p.tpr < need && p.tpr < 256) p.tpr *= 2;
    while (p.tpr * p.nv < need && p.nv < most) p.nv *= 2;
    while (p.tpr * p.nv < need) p.tpr *= 2;
    p.block = p.tpr > 256 ? p.tpr : 256;
    return p;
}

int backward_blocks(long long rows, const RowPlan &p) {
    const long long need = (rows + p.block / p.tpr - 1) / (p.block / p.tpr);
    return (int)(need < kBlocks ? need : kBlocks);
}

// calls f with the plan's V, NV, whether a row spans warps, and the block size as constants
template <typename T, typename F>
void with_plan(const RowPlan &p, F &&f) {
    auto go = [&](auto v, auto most) {
        constexpr int V = decltype(v)::value, M = decltype(most)::value;
        using std::integral_constant;
        integral_constant<int, 256> b256;
        integral_constant<bool, true> big;
        if (p.tpr <= 32)
            f(v, integral_constant<int, 1>{}, integral_constant<bool, false>{}, b256);
        else if (p.nv == 1)
            f(v, integral_constant<int, 1>{}, big, b256);
        else if (p.tpr > 512) {
            if constexpr (V == 1) f(v, most, big, integral_constant<int, 1024>{});
        } else if (p.tpr > 256)
            f(v, most, big, integral_constant<int, 512>{});
        else if (p.nv == M)
            f(v, most, big, b256);
        else if constexpr (M >= 4) {
            if (p.nv == 2)
                f(v, integral_constant<int, 2>{}, big, b256);
            else
                f(v, integral_constant<int, 4>{}, big, b256);
        }
    };
    constexpr int VV = 16 / (int)sizeof(T);
    if (p.v == 1)
        go(std::integral_constant<int, 1>{}, std::integral_constant<int, 8>{});
    else
        go(std::integral_constant<int, VV>{}, std::integral_constant<int, 16 / VV>{});
}

template <typename F>
void with_type(int dtype, F &&f) {
    if (dtype == S4_BF16)
        f(__nv_bfloat16{});
    else if (dtype == S4_F16)
        f(__half{});
    else
        f(float{});
}

bool vector_ok(int dtype, int D, const void *a, const void *b, const void *c) {
    const int elem = dtype == S4_F32 ? 4 : 2;
    return ((size_t)D * elem) % 16 == 0 && (((uintptr_t)a | (uintptr_t)b | (uintptr_t)c) & 15) == 0;
}

}  // namespace

// a partial row of dgamma and dbeta per block
size_t norm_backward_workspace_bytes(int D) { return (size_t)kBlocks * 2 * D * sizeof(float); }

cudaError_t launch_layernorm_rows(int dtype, const void *x, const float *gamma, const float *beta, float eps,
                                  long long rows, int D, void *z, float *mean, float *rstd, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    const RowPlan p = row_plan(D, dtype == S4_F32 ? 4 : 2, vector_ok(dtype, D, x, z, nullptr));
    const int groups = p.block / p.tpr;
    const int grid = (int)((rows + groups - 1) / groups);
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        with_plan<T>(p, [&](auto v, auto nv, auto big, auto most) {
            k_layernorm_rows<T, decltype(v)::value, decltype(nv)::value, decltype(big)::value, decltype(most)::value>
                <<<grid, p.block, 0, st>>>((const T *)x, gamma, beta, eps, rows, D, p.tpr, (T *)z, mean, rstd);
        });
    });
    return cudaGetLastError();
}

cudaError_t launch_layernorm_rows_backward(int dtype, const void *dz, const void *x, const float *gamma,
                                           const float *mean, const float *rstd, long long rows, int D, void *dx,
                                           float *dgamma, float *dbeta, void *ws, cudaStream_t st) {
    const RowPlan p = row_plan(D, dtype == S4_F32 ? 4 : 2, vector_ok(dtype, D, x, dz, dx));
    const int grid = backward_blocks(rows, p);
    // several groups in a block only for tpr <= 128 and one access each: D <= 1024
    const size_t smem = p.block > p.tpr ? (size_t)2 * D * sizeof(float) : 0;
    float *part = (float *)ws;
    if (rows > 0) with_type(dtype, [&](auto t) {   // no rows: zero gradients from no partial rows
        using T = decltype(t);
        with_plan<T>(p, [&](auto v, auto nv, auto big, auto most) {
            k_layernorm_rows_backward<T, decltype(v)::value, decltype(nv)::value, decltype(big)::value,
                                      decltype(most)::value><<<grid, p.block, smem, st>>>(
                (const T *)dz, (const T *)x, gamma, mean, rstd, rows, D, p.tpr, (T *)dx, part);
        });
    });
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    k_sum_partials<<<(2 * D + 31) / 32, 256, 0, st>>>(part, grid, D, dgamma, dbeta);
    return cudaGetLastError();
}

cudaError_t launch_layernorm_channels_backward(const float *dz, const float *x, const float *gamma, float eps,
                                               int Bt, int H, int L, float *dx, float *dgamma, float *dbeta,
                                               void *ws, cudaStream_t st) {
    const long long tiles = (long long)((L + kSteps - 1) / kSteps) * Bt;
    const int grid = (int)(tiles < kBlocks ? tiles : kBlocks);
    float *part = (float *)ws;
    if (H <= 4 * kSlices) {
        k_layernorm_channels_backward_reg<4><<<grid, 256, 0, st>>>(dz, x, gamma, eps, Bt, H, L, dx, part);
    } else if (H <= 16 * kSlices) {
        k_layernorm_channels_backward_reg<16><<<grid, 256, 0, st>>>(dz, x, gamma, eps, Bt, H, L, dx, part);
    } else {
        const int smem = 2 * H * (int)sizeof(float);
        if (smem > 48 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(k_layernorm_channels_backward,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 2 * S4_MAX_BLOCK_H * (int)sizeof(float));
            if (e != cudaSuccess) return e;
        }
        k_layernorm_channels_backward<<<grid, 256, smem, st>>>(dz, x, gamma, eps, Bt, H, L, dx, part);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    k_sum_partials<<<(2 * H + 31) / 32, 256, 0, st>>>(part, grid, H, dgamma, dbeta);
    return cudaGetLastError();
}

}  // namespace s4
