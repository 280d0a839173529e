// norm.cu -- layer norm over token rows (forward and backward) and the
// backward of the S4Block's norm over channels.
//
//   xhat = (x - mu) rstd,  z = xhat gamma + beta,  rstd = (var + eps)^-1/2
//   h = dz gamma,  dx = rstd (h - mean(h) - xhat mean(h xhat))
//   dgamma = sum over rows of dz xhat,  dbeta = sum over rows of dz
//
// Both directions move each array once (rows: forward x -> z, backward x, dz
// -> dx; channels: x, dz -> dx). Measured at 32768 rows of 1024 bf16: forward
// 38 us (3.5 TB/s), backward 49 + 5.5 us (3.7 TB/s). Neither is at a limit: 63
// and 62% of the issue slots, 27 and 41% of DRAM, 23 and 22% of the warps that
// an SM holds (registers), which wait for each other's results and for shared
// memory. 16384 rows of 2048 float, backward: 67 us (6.0 TB/s). Channels, 8 x
// 256 x 16384: 80 us (5.0 TB/s); above 256 channels 2.7 to 3.0 TB/s, see
// there. The weight gradients are summed in registers over all rows a block
// visits (a fixed set, in a fixed order),
// written as one partial row per block and added up by a second small kernel
// in a fixed order: no atomics, the same bits every time.
#include "dtype.cuh"
#include "launch.h"
#include "s4dplr.h"
#include "umma.cuh"

#include <type_traits>

namespace s4 {
namespace {

// Most backward blocks, each with a partial row of weight gradients, on top of
// one bound: no more than are resident. At four per SM throughout, 4096 rows of
// 8192 bf16 ran in two waves (97 us, 59 now), and 32768 of 1024, whose blocks
// are two warps, left the SM half empty (62 and 51 us). Longer rows get fewer
// for the pass over the partial rows: 5.5 us at 1184 of 1024, 6 at 592 of 8192.
int most_blocks(int D) { return 148 * (D <= 512 ? 16 : D <= 2048 ? 8 : 4); }

template <int BYTES>
__device__ __forceinline__ void cp_async(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(umma::saddr(dst)), "l"(src), "n"(BYTES) : "memory");
}

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

// A thread's weights: in registers up to 16 elements, above from L1 where they
// are used. `wide`: the array is 16-byte aligned (D is a multiple of V).
template <int V, int NV>
struct Weights {
    static constexpr bool kKept = V * NV <= 16;
    float kept[kKept ? NV : 1][V];
    const float *w;
    int l, tpr, D;
    bool wide;
    __device__ __forceinline__ Weights(const float *w_, int l_, int tpr_, int D_)
        : w(w_), l(l_), tpr(tpr_), D(D_), wide(V >= 4 && ((size_t)w_ & 15) == 0) {
        if constexpr (kKept)
#pragma unroll
            for (int i = 0; i < NV; ++i) load(i, kept[i]);
    }
    __device__ __forceinline__ void load(int i, float (&o)[V]) const {
        const int c = (l + i * tpr) * V;
        if constexpr (V >= 4) {
            if (wide) {
                if (c < D)
#pragma unroll
                    for (int j = 0; j < V; j += 4) {
                        const float4 f = __ldg(reinterpret_cast<const float4 *>(w + c + j));
                        o[j] = f.x, o[j + 1] = f.y, o[j + 2] = f.z, o[j + 3] = f.w;
                    }
                return;
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < D) o[j] = __ldg(w + c + j);
    }
    __device__ __forceinline__ void get(int i, float (&o)[V]) const {
        if constexpr (kKept) {
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = kept[i][j];
        } else {
            load(i, o);
        }
    }
};

// Rows of 16- or 8-byte packs go through a ring in shared memory: kStages - 1
// rounds of rows are on their way while one is reduced, two rows a round where
// a row takes few packs a thread. A thread copies exactly what it reads, so the
// ring needs no barrier. With the loads in flight in registers they were paid
// for in occupancy (32768 rows of 1024 bf16: forward 86 us a row a block, 49 us
// four rows at a time, 39 us now; backward 74, 117 and 50 us; float rows reach
// 5.2 and 6.0 TB/s). 8-byte packs:
// rows that are multiples of 8 bytes only (30000 of 500 bf16, backward: 30 us,
// as single elements 63). Single elements (V = 1) are loaded where they are used.
constexpr int kStages = 3;
template <int V, int NV, int ARR>
__host__ __device__ constexpr int rows_at_once() { return V > 1 && NV * ARR <= 2 ? 2 : 1; }

// ARR arrays of rows; ring [stage][row][array][NV][thread]
template <typename T, int V, int NV, int ARR>
struct Rows {
    static constexpr int R = rows_at_once<V, NV, ARR>();
    Pack<T, V> *ring;
    const T *src[ARR];
    long long rows;
    int D, l, tpr, stage;

    static size_t bytes(int block) { return V > 1 ? (size_t)kStages * R * ARR * NV * block * V * sizeof(T) : 0; }
    __device__ __forceinline__ Pack<T, V> *slot(int st, int q, int a, int i) const {
        return ring + (((st * R + q) * ARR + a) * NV + i) * (int)blockDim.x + threadIdx.x;
    }
    // rows r .. r + R - 1 into stage st
    __device__ __forceinline__ void fetch(long long r, int st) const {
        if constexpr (V > 1) {
#pragma unroll
            for (int q = 0; q < R; ++q)
                if (r + q < rows)
#pragma unroll
                    for (int a = 0; a < ARR; ++a)
#pragma unroll
                        for (int i = 0; i < NV; ++i) {
                            const int c = (l + i * tpr) * V;
                            if (c >= D) continue;
                            const T *p = src[a] + (r + q) * D + c;
                            if constexpr (V * sizeof(T) == 16)
                                umma::cp_async16(slot(st, q, a, i), p);
                            else
                                cp_async<V * (int)sizeof(T)>(slot(st, q, a, i), p);
                        }
            umma::cp_async_commit();
        }
    }
    // the oldest round has arrived
    __device__ __forceinline__ void wait() const {
        if constexpr (V > 1) asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    }
    // pack i of row r + q, array a, of the current round
    __device__ __forceinline__ void get(long long r, int q, int a, int i, float (&o)[V]) const {
        Pack<T, V> p;
        if constexpr (V > 1)
            p = *slot(stage, q, a, i);
        else
            p.v[0] = src[a][(r + q) * D + l + i * tpr];
        unpack<T, V>(p, o);
    }
    // next round: `stride` rows on
    __device__ __forceinline__ void begin(long long r, long long stride) {
        stage = 0;
#pragma unroll
        for (int k = 0; k + 1 < kStages; ++k) fetch(r + k * stride, k);
    }
    __device__ __forceinline__ void ahead(long long r, long long stride) const {
        fetch(r + (kStages - 1) * stride, stage == 0 ? kStages - 1 : stage - 1);
        wait();
    }
    __device__ __forceinline__ void step() { stage = stage + 1 == kStages ? 0 : stage + 1; }
};

template <typename T, int V, int NV, bool BIG, int MAXT>
__global__ void __launch_bounds__(MAXT) k_layernorm_rows(const T *x, const float *__restrict__ gamma,
                                                         const float *__restrict__ beta, float eps, long long rows,
                                                         int D, int tpr, T *z, float *mean, float *rstd) {
    using L = Rows<T, V, NV, 1>;
    constexpr int R = L::R;
    __shared__ float buf[2 * R * 32];
    extern __shared__ __align__(16) unsigned char ring[];
    int turn = 0;
    const int groups = blockDim.x / tpr, l = threadIdx.x % tpr;
    const long long stride = (long long)gridDim.x * groups * R;
    const float inv = 1.0f / (float)D;
    const Weights<V, NV> ga(gamma, l, tpr, D), be(beta, l, tpr, D);
    L in{reinterpret_cast<Pack<T, V> *>(ring), {x}, rows, D, l, tpr, 0};
    // every group of a block takes the same number of turns (the barrier in group_sum)
    const long long first = (long long)blockIdx.x * groups * R, mine = (threadIdx.x / tpr) * R;
    in.begin(first + mine, stride);
    for (long long r0 = first; r0 < rows; r0 += stride, in.step()) {
        const long long r = r0 + mine;
        in.ahead(r, stride);
        float s[R], mu[R], v[R][NV][V];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            s[q] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (r + q < rows && (l + i * tpr) * V < D)
                    in.get(r, q, 0, i, v[q][i]);
                else
#pragma unroll
                    for (int j = 0; j < V; ++j) v[q][i][j] = 0.0f;
#pragma unroll
                for (int j = 0; j < V; ++j) s[q] += v[q][i][j];
            }
        }
        group_sum<R, BIG>(s, tpr, buf, turn);
#pragma unroll
        for (int q = 0; q < R; ++q) {
            mu[q] = s[q] * inv;
            s[q] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if ((l + i * tpr) * V < D)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        v[q][i][j] -= mu[q];
                        s[q] = fmaf(v[q][i][j], v[q][i][j], s[q]);
                    }
        }
        group_sum<R, BIG>(s, tpr, buf, turn);
        float rs[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            rs[q] = 1.0f / sqrtf(fmaf(s[q], inv, eps));
            if (l == 0 && r + q < rows) {
                mean[r + q] = mu[q];
                rstd[r + q] = rs[q];
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (l + i * tpr) * V;
            if (c >= D) continue;
            float g[V], b[V];
            ga.get(i, g);
            be.get(i, b);
#pragma unroll
            for (int q = 0; q < R; ++q)
                if (r + q < rows) {
                    float o[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) o[j] = fmaf(v[q][i][j] * rs[q], g[j], b[j]);
                    store_pack<T, V>(z + (r + q) * D + c, o);
                }
        }
    }
}

template <typename T, int V, int NV, bool BIG, int MAXT>
__global__ void __launch_bounds__(MAXT) k_layernorm_rows_backward(
    const T *dz, const T *x, const float *__restrict__ gamma, const float *__restrict__ mean,
    const float *__restrict__ rstd, long long rows, int D, int tpr, T *dx, float *part) {
    using L = Rows<T, V, NV, 2>;
    constexpr int R = L::R;
    __shared__ float buf[2 * 2 * R * 32];
    extern __shared__ __align__(16) unsigned char ring[];   // groups > 1: at the end [2][D] floats in its place
    int turn = 0;
    const int groups = blockDim.x / tpr, l = threadIdx.x % tpr, gi = threadIdx.x / tpr;
    float dg[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) dg[i][j] = db[i][j] = 0.0f;
    const Weights<V, NV> ga(gamma, l, tpr, D);
    const float inv = 1.0f / (float)D;
    const long long stride = (long long)gridDim.x * groups * R;
    L in{reinterpret_cast<Pack<T, V> *>(ring), {x, dz}, rows, D, l, tpr, 0};
    float nm[R], nr[R];
    auto stats = [&](long long r) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            nm[q] = r + q < rows ? __ldg(mean + r + q) : 0.0f;
            nr[q] = r + q < rows ? __ldg(rstd + r + q) : 0.0f;
        }
    };
    // every group of a block takes the same number of turns (the barrier in group_sum)
    const long long first = (long long)blockIdx.x * groups * R, mine = gi * R;
    in.begin(first + mine, stride);
    stats(first + mine);
    for (long long r0 = first; r0 < rows; r0 += stride, in.step()) {
        const long long r = r0 + mine;
        in.ahead(r, stride);
        float s[2 * R], mu[R], rs[R], xh[R][NV][V], h[R][NV][V];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            s[2 * q] = s[2 * q + 1] = 0.0f;
            mu[q] = nm[q];
            rs[q] = nr[q];
            if (r + q < rows)
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if ((l + i * tpr) * V < D) {
                        float g[V];
                        ga.get(i, g);
                        in.get(r, q, 0, i, xh[q][i]);
                        in.get(r, q, 1, i, h[q][i]);
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float d = h[q][i][j], x = (xh[q][i][j] - mu[q]) * rs[q];
                            dg[i][j] = fmaf(d, x, dg[i][j]);
                            db[i][j] += d;
                            xh[q][i][j] = x;
                            h[q][i][j] = d * g[j];
                            s[2 * q] += h[q][i][j];
                            s[2 * q + 1] = fmaf(h[q][i][j], x, s[2 * q + 1]);
                        }
                    }
        }
        stats(r + stride);
        group_sum<2 * R, BIG>(s, tpr, buf, turn);
#pragma unroll
        for (int q = 0; q < R; ++q) {
            if (r + q >= rows) continue;
            const float m0 = s[2 * q] * inv, m1 = s[2 * q + 1] * inv;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (l + i * tpr) * V;
                if (c < D) {
                    if constexpr (sizeof(T) == 4) {   // read again: nothing to convert, and registers are short
                        float g[V];
                        ga.get(i, g);
                        in.get(r, q, 0, i, xh[q][i]);
                        in.get(r, q, 1, i, h[q][i]);
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            xh[q][i][j] = (xh[q][i][j] - mu[q]) * rs[q];
                            h[q][i][j] *= g[j];
                        }
                    }
                    float o[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) o[j] = rs[q] * (h[q][i][j] - fmaf(xh[q][i][j], m1, m0));
                    store_pack<T, V>(dx + (r + q) * D + c, o);
                }
            }
        }
    }
    float *sacc = reinterpret_cast<float *>(ring);
    if (groups > 1) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();   // the ring is used up
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

// out0[c], out1[c] = sums over n partial rows [2][D]: 32 columns a block, 32
// strided slices of the rows each, added in order
__global__ void __launch_bounds__(1024) k_sum_partials(const float *__restrict__ part, int n, int D, float *out0,
                                                       float *out1) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, w = threadIdx.x >> 5;
    float a = 0.0f;
    if (c < 2 * D) {
#pragma unroll 8
        for (int r = w; r < n; r += 32) a += part[(size_t)r * 2 * D + c];
    }
    s[w][lane] = a;
    __syncthreads();
    if (w == 0 && c < 2 * D) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += s[i][lane];
        if (c < D)
            out0[c] = t;
        else
            out1[c - D] = t;
    }
}

// ---------------------------------------------------- channel layout ------
// x, dz [Bt, H, L]: a tile is some time steps of one batch row, W threads x 4
// steps wide and 16 slices of the channels deep.
constexpr int kSlices = 16;

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
template <int W>
__device__ __forceinline__ float4 slice_sum(float4 a, float4 (*red)[W], int hs, int tl) {
    __syncthreads();
    red[hs][tl] = a;
    __syncthreads();
    float4 s = red[0][tl];
#pragma unroll
    for (int i = 1; i < kSlices; ++i) s = add4(s, red[i][tl]);
    return s;
}
// sum over the W threads of a slice
template <int W>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of N values per step over all channels, for 256 threads as 32 slices of
// 8: within a warp by shuffles, then the eight warps' through shared memory, one
// barrier, two buffers in turn.
template <int N>
__device__ __forceinline__ void step_sums(float4 (&a)[N], float4 (*red)[3][8][8], int &turn) {
    const int lane = threadIdx.x & 31, tl = lane & 7, w = threadIdx.x >> 5;
    float4 (*b)[8][8] = red[turn++ & 1];
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int o = 8; o < 32; o <<= 1)
            a[n] = add4(a[n], make_float4(__shfl_xor_sync(0xffffffffu, a[n].x, o), __shfl_xor_sync(0xffffffffu, a[n].y, o),
                                          __shfl_xor_sync(0xffffffffu, a[n].z, o), __shfl_xor_sync(0xffffffffu, a[n].w, o)));
        if (lane < 8) b[n][w][tl] = a[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        a[n] = b[n][0][tl];
#pragma unroll
        for (int k = 1; k < 8; ++k) a[n] = add4(a[n], b[n][k][tl]);
    }
}

// H <= 32 NV: tiles of 32 steps. Three tiles of x and dz are in shared memory
// or on their way to it (a thread copies exactly what it reads, so a copy needs
// no barrier), so that loads go on while a tile is reduced: with the loads of a
// tile in registers behind each other's reductions the memory idled half the
// time (8 x 256 x 16384: 109 us; now 82 us, 4.9 TB/s). The weight gradients of
// a thread's channels stay in registers over all tiles of the block.
constexpr int kChStages = 3;

template <int NV>
__global__ void __launch_bounds__(256) k_layernorm_channels_backward_reg(
    const float *__restrict__ dz, const float *__restrict__ x, const float *__restrict__ gamma, float eps, int Bt,
    int H, int L, float *dx, float *part) {
    __shared__ float4 red[2][3][8][8];
    extern __shared__ __align__(16) float4 tiles_s[];   // [stages][x, dz][H][8]
    constexpr int W = 8, kSteps = 4 * W;
    const int tl = threadIdx.x % W, hs = threadIdx.x / W;
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float inv = 1.0f / (float)H;
    float dg[NV], db[NV], ga[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        dg[i] = db[i] = 0.0f;
        ga[i] = hs + 32 * i < H ? __ldg(gamma + hs + 32 * i) : 0.0f;
    }
    const unsigned tiles_l = (L + kSteps - 1) / kSteps;
    const long long tiles = (long long)tiles_l * Bt;
    int turn = 0;
    auto place = [&](long long tile, int &t) {   // the thread's first element of a tile, and its first step
        const long long b = tile / tiles_l;
        t = (int)(tile - b * tiles_l) * kSteps + 4 * tl;
        return (size_t)b * H * L + t;
    };
    auto fetch = [&](long long tile, int st) {
        int t;
        if (tile < tiles) {
            const size_t base = place(tile, t);
            float4 *s = tiles_s + (size_t)st * 2 * H * W + tl;
            if (t < L)   // L is a multiple of 16: t < L implies t + 3 < L
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int h = hs + 32 * i;
                    if (h < H) {
                        umma::cp_async16(s + h * W, x + base + (size_t)h * L);
                        umma::cp_async16(s + (H + h) * W, dz + base + (size_t)h * L);
                    }
                }
        }
        umma::cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k + 1 < kChStages; ++k) fetch(blockIdx.x + (long long)k * gridDim.x, k);
    int st = 0;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        fetch(tile + (long long)(kChStages - 1) * gridDim.x, st == 0 ? kChStages - 1 : st - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kChStages - 1) : "memory");   // this tile's are the oldest
        int t;
        const size_t base = place(tile, t);
        const bool in = t < L;
        const float4 *sx = tiles_s + (size_t)st * 2 * H * W + tl;
        st = st + 1 == kChStages ? 0 : st + 1;
        float4 v[NV], w[NV], a[2] = {zero, zero}, s[2] = {zero, zero};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int h = hs + 32 * i;
            const bool ok = in && h < H;
            v[i] = ok ? sx[h * W] : zero;
            w[i] = ok ? sx[(H + h) * W] : zero;
            a[0] = add4(a[0], v[i]);
            a[1] = add4(a[1], scale4(w[i], ga[i]));
            db[i] += sum4(w[i]);   // steps past L hold dz = 0
        }
        step_sums<2>(a, red, turn);
        const float4 mu = scale4(a[0], inv), m0 = scale4(a[1], inv);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (hs + 32 * i < H) {
                v[i] = sub4(v[i], mu);
                s[0] = fma4(v[i], v[i], s[0]);
                s[1] = fma4(scale4(w[i], ga[i]), v[i], s[1]);
            }
        step_sums<2>(s, red, turn);
        const float4 rs = rstd4(s[0], inv, eps);
        const float4 m1 = mul4(scale4(s[1], inv), mul4(rs, rs));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int h = hs + 32 * i;
            if (h < H) {
                dg[i] += sum4(mul4(w[i], mul4(v[i], rs)));
                if (in)
                    *reinterpret_cast<float4 *>(dx + base + (size_t)h * L) =
                        mul4(rs, sub4(scale4(w[i], ga[i]), fma4(v[i], m1, m0)));
            }
        }
    }
    float *p = part + (size_t)blockIdx.x * 2 * H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int h = hs + 32 * i;
        const float g = lane_sum<W>(dg[i]), b = lane_sum<W>(db[i]);
        if (h < H && tl == 0) {
            p[h] = g;
            p[H + h] = b;
        }
    }
}

// any H: the tile is read three times (mean; variance and the two sums of the
// gradient; output), dz twice, and the weight gradients are kept in shared
// memory, each channel's by the slice that owns it. The tiles under way at once
// are larger than L2 from some 400 channels on (4 blocks an SM, 512 H bytes
// each), then every read comes from memory: at 4 x 1024 x 8192 670 MB read for
// 268, 0.2% of them found in L2, 65% of DRAM's rate, the rest waiting for loads
// that are not started ahead. Measured: 8 x 512 x 16384 300 us, 32 x 1024 x 8192
// 1076 us, 2.7 and 3.0 TB/s of the 12 bytes an element that have to move; 2 x
// 4096 x 4096, with 128 tiles fewer blocks than SMs, 429 us.
__global__ void __launch_bounds__(256) k_layernorm_channels_backward(
    const float *__restrict__ dz, const float *__restrict__ x, const float *__restrict__ gamma, float eps, int Bt,
    int H, int L, float *dx, float *part) {
    constexpr int W = 16, kSteps = 4 * W;
    __shared__ float4 red[kSlices][W];
    extern __shared__ float sacc[];   // [2][H]
    const int tl = threadIdx.x % (W), hs = threadIdx.x / (W);
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
        const float4 mu = scale4(slice_sum<W>(a, red, hs, tl), inv);
        float4 ss = zero, s0 = zero, s1 = zero;
        if (in)
            for (int h = hs; h < H; h += kSlices) {
                const float4 c = sub4(*reinterpret_cast<const float4 *>(x + base + (size_t)h * L), mu);
                const float4 w = scale4(*reinterpret_cast<const float4 *>(dz + base + (size_t)h * L), __ldg(gamma + h));
                ss = fma4(c, c, ss);
                s0 = add4(s0, w);
                s1 = fma4(w, c, s1);
            }
        const float4 rs = rstd4(slice_sum<W>(ss, red, hs, tl), inv, eps);
        const float4 m0 = scale4(slice_sum<W>(s0, red, hs, tl), inv);
        const float4 m1 = mul4(scale4(slice_sum<W>(s1, red, hs, tl), inv), rs);
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
            g = lane_sum<W>(g);
            b = lane_sum<W>(b);
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
// threads, at most kElements elements a thread (8 when single). Fewer threads
// make a row's reductions and addresses cost fewer warps; 32 elements a thread
// leave too few warps for their registers (16384 rows of 2048, forward: 41 us
// bf16 and 64 us float, 38 and 52 with 16; backward at 32, 1024 bf16: 97 us).
constexpr int kElements = 16;
struct RowPlan { int v, nv, tpr, block; };

RowPlan row_plan(int D, int elem, int bytes, int elements) {
    RowPlan p;
    p.v = bytes / elem;
    const int need = (D + p.v - 1) / p.v, most = elements / p.v < 8 ? elements / p.v : 8;
    p.nv = 1;
    p.tpr = 1;
    while (p.tpr < need && p.tpr < 32) p.tpr *= 2;
    while (p.tpr * p.nv < need && p.nv < most) p.nv *= 2;
    while (p.tpr * p.nv < need) p.tpr *= 2;   // D <= 8192: at most 512 threads, 1024 with single elements
    // rows of more than a warp have a block each, whose barrier nobody else waits at
    p.block = p.tpr > 32 ? p.tpr : 256;
    return p;
}

// blocks for `rows` rows, at most `most`
int row_blocks(long long rows, const RowPlan &p, int at_once, int most) {
    const int per = p.block / p.tpr * at_once;
    const long long need = (rows + per - 1) / per;
    return (int)(need < most ? need : most);
}

// calls f with the plan's V, NV, whether a row spans warps, and the largest block as constants
template <typename T, int ELEMENTS, typename F>
void with_plan(const RowPlan &p, F &&f) {
    using std::integral_constant;
    auto go = [&](auto v, auto most) {
        constexpr int V = decltype(v)::value, M = decltype(most)::value;
        integral_constant<int, 256> b256;
        if (p.tpr > 256) {
            f(v, most, integral_constant<bool, true>{}, integral_constant<int, V == 1 ? 1024 : 512>{});
        } else if (p.tpr > 32) {
            f(v, most, integral_constant<bool, true>{}, b256);
        } else {
            integral_constant<bool, false> small;
            if (p.nv == 1)
                f(v, integral_constant<int, 1>{}, small, b256);
            else if (p.nv == 2)
                f(v, integral_constant<int, 2>{}, small, b256);
            else if constexpr (M >= 4) {
                if (p.nv == 4) return f(v, integral_constant<int, 4>{}, small, b256);
                if constexpr (M >= 8) f(v, integral_constant<int, 8>{}, small, b256);
            }
        }
    };
    constexpr int VV = 16 / (int)sizeof(T);
    constexpr int HALF = ELEMENTS / (VV / 2);
    if (p.v == 1)
        go(integral_constant<int, 1>{}, integral_constant<int, 8>{});
    else if (p.v == VV / 2)
        go(integral_constant<int, VV / 2>{}, integral_constant<int, HALF < 8 ? HALF : 8>{});
    else
        go(integral_constant<int, VV>{}, integral_constant<int, ELEMENTS / VV>{});
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

// bytes of an access: 16, 8 or one element, whatever rows and addresses are multiples of
int access_bytes(int dtype, int D, const void *a, const void *b, const void *c) {
    const int elem = dtype == S4_F32 ? 4 : 2;
    const size_t all = ((size_t)D * elem) | (uintptr_t)a | (uintptr_t)b | (uintptr_t)c;
    return all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : elem;
}

}  // namespace

// a partial row of dgamma and dbeta per block
size_t norm_backward_workspace_bytes(int D) { return (size_t)most_blocks(D) * 2 * D * sizeof(float); }

cudaError_t launch_layernorm_rows(int dtype, const void *x, const float *gamma, const float *beta, float eps,
                                  long long rows, int D, void *z, float *mean, float *rstd, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    const RowPlan p = row_plan(D, dtype == S4_F32 ? 4 : 2, access_bytes(dtype, D, x, z, nullptr), kElements);
    cudaError_t err = cudaSuccess;
    with_type(dtype, [&](auto t) {
        using T = decltype(t);
        with_plan<T, kElements>(p, [&](auto v, auto nv, auto big, auto most) {
            constexpr int V = decltype(v)::value, NV = decltype(nv)::value, MAXT = decltype(most)::value;
            static Resident resident;
            static SmemLimit limit;
            auto *kernel = k_layernorm_rows<T, V, NV, decltype(big)::value, MAXT>;
            const size_t smem = Rows<T, V, NV, 1>::bytes(p.block);
            err = limit.raise(kernel, smem);
            if (err != cudaSuccess) return;
            const int grid = row_blocks(rows, p, rows_at_once<V, NV, 1>(), 148 * resident.of(kernel, p.block, smem));
            kernel<<<grid, p.block, smem, st>>>((const T *)x, gamma, beta, eps, rows, D, p.tpr, (T *)z, mean, rstd);
        });
    });
    return err != cudaSuccess ? err : cudaGetLastError();
}

cudaError_t launch_layernorm_rows_backward(int dtype, const void *dz, const void *x, const float *gamma,
                                           const float *mean, const float *rstd, long long rows, int D, void *dx,
                                           float *dgamma, float *dbeta, void *ws, cudaStream_t st) {
    const RowPlan p = row_plan(D, dtype == S4_F32 ? 4 : 2, access_bytes(dtype, D, x, dz, dx), kElements);
    int grid = 0;
    // several groups in a block only for tpr <= 32: D <= 1024
    const size_t acc = p.block > p.tpr ? (size_t)2 * D * sizeof(float) : 0;
    cudaError_t err = cudaSuccess;
    float *part = (float *)ws;
    if (rows > 0) with_type(dtype, [&](auto t) {   // no rows: zero gradients from no partial rows
        using T = decltype(t);
        with_plan<T, kElements>(p, [&](auto v, auto nv, auto big, auto most) {
            constexpr int V = decltype(v)::value, NV = decltype(nv)::value, MAXT = decltype(most)::value;
            static Resident resident;
            static SmemLimit limit;
            auto *kernel = k_layernorm_rows_backward<T, V, NV, decltype(big)::value, MAXT>;
            const size_t ring = Rows<T, V, NV, 2>::bytes(p.block), smem = ring > acc ? ring : acc;
            err = limit.raise(kernel, smem);
            if (err != cudaSuccess) return;
            const int fit = 148 * resident.of(kernel, p.block, smem);
            grid = row_blocks(rows, p, rows_at_once<V, NV, 2>(), fit < most_blocks(D) ? fit : most_blocks(D));
            kernel<<<grid, p.block, smem, st>>>(
                (const T *)dz, (const T *)x, gamma, mean, rstd, rows, D, p.tpr, (T *)dx, part);
        });
    });
    if (err != cudaSuccess) return err;
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    k_sum_partials<<<(2 * D + 31) / 32, 1024, 0, st>>>(part, grid, D, dgamma, dbeta);
    return cudaGetLastError();
}

cudaError_t launch_layernorm_channels_backward(const float *dz, const float *x, const float *gamma, float eps,
                                               int Bt, int H, int L, float *dx, float *dgamma, float *dbeta,
                                               void *ws, cudaStream_t st) {
    // tiles of 32 steps through shared memory up to 256 channels, of 64 steps read three times above
    const bool staged = H <= 256;
    const int steps = staged ? 32 : 64;
    const long long tiles = (long long)((L + steps - 1) / steps) * Bt;
    float *part = (float *)ws;
    const int blocks = 148 * 4;
    int grid = (int)(tiles < blocks ? tiles : blocks);
    if (staged) {
        const int smem = kChStages * 2 * H * 128, most = 148 * (smem > 100 * 1024 ? 1 : smem > 50 * 1024 ? 2 : 4);
        grid = (int)(tiles < most ? tiles : most);
        auto go = [&](auto *f) {
            if (smem > 40 * 1024) {
                cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kChStages * 65536);
                if (e != cudaSuccess) return e;
            }
            f<<<grid, 256, smem, st>>>(dz, x, gamma, eps, Bt, H, L, dx, part);
            return cudaSuccess;
        };
        cudaError_t e = H <= 64 ? go(k_layernorm_channels_backward_reg<2>)
                                : H <= 128 ? go(k_layernorm_channels_backward_reg<4>)
                                           : go(k_layernorm_channels_backward_reg<8>);
        if (e != cudaSuccess) return e;
    } else {
        const int smem = 2 * H * (int)sizeof(float);
        if (smem > 40 * 1024) {   // with the static 4 KB above the 48 KB that need no asking
            cudaError_t e = cudaFuncSetAttribute(k_layernorm_channels_backward,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 2 * S4_MAX_BLOCK_H * (int)sizeof(float));
            if (e != cudaSuccess) return e;
        }
        k_layernorm_channels_backward<<<grid, 256, smem, st>>>(dz, x, gamma, eps, Bt, H, L, dx, part);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    k_sum_partials<<<(2 * H + 31) / 32, 1024, 0, st>>>(part, grid, H, dgamma, dbeta);
    return cudaGetLastError();
}

}  // namespace s4
