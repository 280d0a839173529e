// delta_prep.cu -- the part of the chunked gated delta rule that does not
// depend on the state: for every chunk and value head the images of
// T = (I + A D_b)^-1 and PT = P D_b T and the gates' factors.
//
// One block per chunk and value head. [K; Q] K^T is one M = 128 product (rows
// 0-63 give A, rows 64-127 give P); two threads share a row of the
// accumulator. T is inverted in float: the 16 x 16 diagonal blocks by forward
// substitution, a column a thread, then T21 = -T22 A21 T11 twice, for blocks of
// 16 and of 32. PT is a second product with P as operand in tensor memory.
// Bound by the latency of these steps one after the other: four blocks of
// eight warps share an SM (128 tensor-memory columns each). Measured: 4 x 4096
// tokens, 32 heads of 128 bf16 (8192 blocks) 250 us, 18 us a wave of blocks;
// 41% of the issue slots, the rest waits at barriers. With four warps a block
// and 1 x 4 products it was 289 us.
#include "delta.cuh"
#include "s4dplr.h"

namespace s4 {
namespace {

using namespace delta;

constexpr int kLd = kC + 4;   // row stride of the float matrices: 16-byte rows, shifted banks
constexpr int kMat = kC * kLd * 4;
constexpr int kTImg = kC * kC * 2;   // one part of T, 64 x 64

// where row r of T (pt = 0) or PT (1), column group cg of a packed part lies; r / 16 >= cg / 2
__device__ __forceinline__ int packed(int r, int cg, int pt) {
    const int ks = cg >> 1, pr = r - 16 * ks;
    return tp_offset(ks) + (cg & 1) * tp_group(ks) + pt * tp_rows(ks) + (pr >> 3) * 128 + (pr & 7) * 16;
}

// Shared memory: the images of [K; Q], in whose place T (float) and behind it
// T's parts come later; A D_b (float) behind the images, which the parts may
// overwrite when T is done.
template <typename T, int DKT>
struct PrepSmem {
    static constexpr int kImg = kq_bytes<T, DKT>() > kMat ? kq_bytes<T, DKT>() : kMat;
    static constexpr int kParts = kMat + 3 * kTImg;
    static constexpr int kBig = kImg + kMat > kParts ? kImg + kMat : kParts;
    static constexpr int kBytes = kBig + 6 * kC * 4 + 64;
};

// put(row, column, 4 values) for +-X Z, N x N float matrices of row stride kLd, by
// the first N * N / 8 of the threads, 2 x 4 values each (of 1, 2 and 4 rows a
// thread the least time: more rows load less, but fewer warps wait longer)
template <int N, bool NEG, typename F>
__device__ __forceinline__ void small_product(const float *X, const float *Z, int t, F &&put) {
    if (t >= N * N / 8) return;
    const int r0 = t / (N / 4) * 2, c = t % (N / 4) * 4;
    float y[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) y[i][j] = 0.0f;
#pragma unroll
    for (int k = 0; k < N; k += 4) {
        float x[2][4], z[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 w = *reinterpret_cast<const float4 *>(Z + (k + i) * kLd + c);
            z[i][0] = w.x, z[i][1] = w.y, z[i][2] = w.z, z[i][3] = w.w;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 u = *reinterpret_cast<const float4 *>(X + (r0 + i) * kLd + k);
            x[i][0] = u.x, x[i][1] = u.y, x[i][2] = u.z, x[i][3] = u.w;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) y[i][j] = fmaf(NEG ? -x[i][q] : x[i][q], z[q][j], y[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) put(r0 + i, c, make_float4(y[i][0], y[i][1], y[i][2], y[i][3]));
}

template <typename T, int DKT>
__global__ void __launch_bounds__(256, PrepSmem<T, DKT>::kBytes < 57000 ? 4 : PrepSmem<T, DKT>::kBytes < 76000 ? 3 : 2)
    k_delta_prep(DeltaArgs a, unsigned char *ws, unsigned char *images, unsigned *flags) {
    using L = PrepSmem<T, DKT>;
    constexpr int NB = Parts<T>::n, kPart = 2 * kC * DKT * 2;
    extern __shared__ __align__(1024) unsigned char smem[];
    float *Ts = reinterpret_cast<float *>(smem), *As = reinterpret_cast<float *>(smem + L::kImg);
    unsigned char *parts = smem + kMat;
    // G / ln 2 as a float and what it leaves out: differences of large sums keep float's accuracy
    float2 *Gs = reinterpret_cast<float2 *>(smem + L::kBig);
    float *cs = reinterpret_cast<float *>(Gs + kC), *bs = cs + kC, *ds = bs + kC, *rs = ds + kC;
    uint64_t *bar = reinterpret_cast<uint64_t *>(rs + kC);
    uint64_t *done = bar + 1;   // for the block's end
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + 2);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

    const long long slot = blockIdx.x / a.hv;
    const int hv = blockIdx.x % a.hv, per = a.hv / a.hk, hk = hv / per;
    const Chunk ch = chunk_of(a, slot);
    if (ch.rows <= 0) return;   // a slot no chunk uses
    const int rows = ch.rows;
    const long long tok = ch.tok;

    load_image<T, DKT>(smem, kPart, 2048, (const T *)a.k + tok * a.sk + (long long)hk * a.dk, a.sk, rows, a.dk, warp, 8);
    load_image<T, DKT>(smem + 1024, kPart, 2048, (const T *)a.q + tok * a.sq + (long long)hk * a.dk, a.sq, rows, a.dk,
                       warp, 8);
    if (warp == 0) umma::tmem_alloc(tslot, 128);
    if (tid == 0) {
        umma::mbar_init(bar, 1);
        umma::mbar_init(done, 1);
        umma::fence_mbar_init();
    }
    if (warp == 1) {
        const GateSums gt = gate_sums(a, tok, hv, rows, lane);
        const int j = 2 * lane;
        const double x = gt.x, y = gt.y;
        const float b0 = gt.b0, b1 = gt.b1;
        const float xf = (float)x, yf = (float)y;
        Gs[j] = make_float2(xf, (float)(x - xf));
        Gs[j + 1] = make_float2(yf, (float)(y - yf));
        bs[j] = b0;
        bs[j + 1] = b1;
        // beta_j e^(G at the end of j's 16 tokens - G_j); the factor e^(G_i - G at that end) is the row's
        const double end = __shfl_sync(0xffffffffu, y, lane | 7), all = __shfl_sync(0xffffffffu, y, 31);
        cs[j] = b0 * exp2f((float)(end - x));
        cs[j + 1] = b1 * exp2f((float)(end - y));
        // within the 16 tokens: from G of their first, while both factors are far from float's limits (2^60)
        const double first = __shfl_sync(0xffffffffu, x, lane & 24);
        const bool near = first - end < 60.0;
        rs[j] = near ? exp2f((float)(x - first)) : -1.0f;
        rs[j + 1] = near ? exp2f((float)(y - first)) : -1.0f;
        ds[j] = b0 * exp2f((float)(near ? first - x : 0.0));
        ds[j + 1] = b1 * exp2f((float)(near ? first - y : 0.0));
        float *fac = reinterpret_cast<float *>(ws + (size_t)blockIdx.x * kUnitBytes + kTpBytes);
        *reinterpret_cast<float2 *>(fac + j) = make_float2(exp2f(xf), exp2f(yf));
        *reinterpret_cast<float2 *>(fac + kC + j) =
            make_float2(b0 * exp2f((float)(all - x)), b1 * exp2f((float)(all - y)));
    }
    umma::cp_async_commit();
    umma::cp_async_wait_all();
    umma::fence_proxy_async();
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tm = uniform(*tslot), base = saddr(smem);
    bool ok = true;
    if (warp == 0) {
        if (elect()) {
            bool acc = false;
#pragma unroll
            for (int o = 2; o >= 0; --o)   // parts' products, the smallest first
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int j = o - i;
                    if (j < 0 || j >= NB) continue;
#pragma unroll
                    for (int ks = 0; ks < DKT / 16; ++ks) {
                        umma::mma_bf16(tm, desc_k(base + i * kPart + ks * 4096, 2048, 128),
                                       desc_k(base + j * kPart + ks * 4096, 2048, 128), idesc(kC, false, false), acc);
                        acc = true;
                    }
                }
            umma::commit(bar);
        }
        __syncwarp();
    }
    if (hv % per == 0) {   // the images for the chains (a bulk store would keep this memory busy for longer)
        uint4 *dst = reinterpret_cast<uint4 *>(images + (size_t)(slot * a.hk + hk) * kq_bytes<T, DKT>());
#pragma unroll 4
        for (int n = tid; n < kq_bytes<T, DKT>() / 16; n += 256) dst[n] = reinterpret_cast<const uint4 *>(smem)[n];
    }
    try_wait(ok, bar, 0);
    umma::fence_after_sync();
    const uint32_t mine = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const int i = tid & (kC - 1), ib = i >> 4;   // this thread's row, and its 16 tokens
    const bool is_p = warp & 2;                  // of P, or of A
    const int half = warp >> 2;                  // of the columns
    const float mul = is_p ? a.scale : 1.0f;
    {
        const float2 Gi = Gs[i];
        auto decay = [&](int j) {   // e^(G_i - G_j)
            const float2 Gj = Gs[j];
            return exp2f((Gi.x - Gj.x) + (Gi.y - Gj.y));
        };
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int c = 32 * half + 16 * n;
            float d[16];
            if (c / 16 > (i | 31) >> 4) {   // above the diagonal for the whole warp
                if (is_p) {
                    const uint32_t z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                    tm_st8(mine + c, z);
                    tm_st8(mine + c + 8, z);
                    tm_st8(mine + 64 + c / 2, z);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4 *>(As + i * kLd + c + j) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
                continue;
            }
            tm_ld16(mine + c, d);
            if (c / 16 < ib) {   // all columns are earlier tokens: one factor for the row, one for each column
                const float rf = mul * decay(c + 15);
                float e[16];
                get16(cs + c, e);
#pragma unroll
                for (int j = 0; j < 16; ++j) d[j] *= rf * e[j];
            } else if (c / 16 == ib) {
                const int m = is_p ? i + 1 : i;
                const float rf = rs[i];
                if (rf >= 0.0f) {   // the same for the 16 tokens
                    float e[16];
                    get16(ds + c, e);
#pragma unroll
                    for (int j = 0; j < 16; ++j) d[j] = c + j < m ? d[j] * (mul * rf * e[j]) : 0.0f;
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) d[j] = c + j < m ? d[j] * (mul * bs[c + j]) * decay(c + j) : 0.0f;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) d[j] = 0.0f;
            }
            if (!is_p) {
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<float4 *>(As + i * kLd + c + j) = make_float4(d[j], d[j + 1], d[j + 2], d[j + 3]);
            } else {   // P as operand; what its rows 0-63 hold only meets results that go unread
                tm_split16(mine + c, mine + 64 + c / 2, d);
            }
        }
        tm_wait_st();
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp < 4) {   // the 16 x 16 diagonal blocks of T by columns, a warp each: x_r = [r = c] - sum_{j < r} A_rj x_j
        const int o = 16 * warp, c = lane & 15;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float acc[4] = {r == c ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < r; j += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(As + (o + r) * kLd + o + j);
                acc[0] = fmaf(-v.x, x[j], acc[0]);
                if (j + 1 < r) acc[1] = fmaf(-v.y, x[j + 1], acc[1]);
                if (j + 2 < r) acc[2] = fmaf(-v.z, x[j + 2], acc[2]);
                if (j + 3 < r) acc[3] = fmaf(-v.w, x[j + 3], acc[3]);
            }
            x[r] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
        }
        if (lane < 16)
#pragma unroll
            for (int r = 0; r < 16; ++r) Ts[(o + r) * kLd + o + c] = x[r];
    }
    __syncthreads();
    // T21 = -T22 (A21 T11), first for the two pairs of 16 x 16 blocks, then for
    // the 32 x 32 ones; A21 T11 goes where A12 = 0 lies
    {
        const int o = 32 * half, t = tid & 127;
        small_product<16, false>(As + (o + 16) * kLd + o, Ts + o * kLd + o, t, [&](int r, int c, float4 y) {
            *reinterpret_cast<float4 *>(As + (o + r) * kLd + o + 16 + c) = y;
        });
        __syncthreads();
        small_product<16, true>(Ts + (o + 16) * kLd + o + 16, As + o * kLd + o + 16, t,
                                        [&](int r, int c, float4 y) {
                                            *reinterpret_cast<float4 *>(Ts + (o + 16 + r) * kLd + o + c) = y;
                                            *reinterpret_cast<float4 *>(Ts + (o + r) * kLd + o + 16 + c) =
                                                make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                                        });
    }
    __syncthreads();
    small_product<32, false>(As + 32 * kLd, Ts, tid, [&](int r, int c, float4 y) {
        *reinterpret_cast<float4 *>(As + r * kLd + 32 + c) = y;
    });
    __syncthreads();
    small_product<32, true>(Ts + 32 * kLd + 32, As + 32, tid, [&](int r, int c, float4 y) {
        *reinterpret_cast<float4 *>(Ts + (32 + r) * kLd + c) = y;
    });
    __syncthreads();
    unsigned char *out = ws + (size_t)blockIdx.x * kUnitBytes;
    {   // T's parts: into shared memory as operand and to the workspace
        const int r = tid & 63;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int cg = (tid >> 6) + 4 * n;
            uint32_t w[4][3];
            const bool in = cg <= r / 8;   // the lower triangle; columns behind the diagonal's block are not read above it
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f), y = x;
            if (8 * cg > (r | 31)) {   // above the diagonal for the whole warp
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    *reinterpret_cast<uint4 *>(parts + q * kTImg + (r >> 3) * 128 + cg * 1024 + (r & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                continue;
            }
            if (in) {
                x = *reinterpret_cast<const float4 *>(Ts + r * kLd + 8 * cg);
                y = *reinterpret_cast<const float4 *>(Ts + r * kLd + 8 * cg + 4);
                if (cg == r / 8) {   // zeros above the diagonal
                    float z[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[j] = j <= (r & 7) ? z[j] : 0.0f;
                    x = make_float4(z[0], z[1], z[2], z[3]);
                    y = make_float4(z[4], z[5], z[6], z[7]);
                }
            }
            split<3>(x.x, x.y, w[0]);
            split<3>(x.z, x.w, w[1]);
            split<3>(y.x, y.y, w[2]);
            split<3>(y.z, y.w, w[3]);
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const uint4 v = make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
                *reinterpret_cast<uint4 *>(parts + q * kTImg + (r >> 3) * 128 + cg * 1024 + (r & 7) * 16) = v;
                if (r / 16 >= cg / 2) *reinterpret_cast<uint4 *>(out + q * kTpImage + packed(r, cg, 0)) = v;
            }
        }
    }
    umma::fence_proxy_async();
    // PT = P T, K over T's rows, 32 columns at a time (rows 32 and up for the
    // second half), so that P's parts and the result share 128 columns
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        umma::fence_before_sync();
        __syncthreads();
        umma::fence_after_sync();
        if (warp == 0) {
            if (elect()) {
                bool acc = false;
#pragma unroll
                for (int o = 2; o >= 0; --o)
#pragma unroll
                    for (int p = 0; p <= o; ++p)
#pragma unroll
                        for (int ks = 2 * pass; ks < kC / 16; ++ks) {
                            mma_ts(tm + 96, tm + (p < 2 ? 16 * ks + 8 * p : 64 + 8 * ks),
                                   desc_mn(saddr(parts) + (o - p) * kTImg + ks * 256 + pass * 4096, 128, 1024),
                                   idesc(32, false, true), acc);
                            acc = true;
                        }
                umma::commit(bar);
            }
            __syncwarp();
        }
        try_wait(ok, bar, 1 ^ pass);
        umma::fence_after_sync();
        if (is_p) {
            float d[16];
            tm_ld16(mine + 96 + 16 * half, d);
            const int c = 32 * pass + 16 * half;
            if (ib >= c / 16)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[4][3];
#pragma unroll
                    for (int j = 0; j < 4; ++j) split<3>(d[8 * h + 2 * j], d[8 * h + 2 * j + 1], w[j]);
#pragma unroll
                    for (int q = 0; q < 3; ++q)
                        *reinterpret_cast<uint4 *>(out + q * kTpImage + packed(i, c / 8 + h, 1)) =
                            make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
                }
        }
    }
    if (!ok && flags) atomicOr(flags, S4_FLAG_TIMEOUT);
    if (warp == 0 && !all_ok(ok)) {   // the products' own warp has not seen the last ones done
        if (elect()) umma::commit(done);
        __syncwarp();
        umma::mbar_wait(done, 0, kDrainLimit);
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 0) umma::tmem_dealloc(tm, 128);
}

template <typename T, int DKT>
cudaError_t run(const DeltaArgs &a, void *ws, unsigned *flags, cudaStream_t st) {
    constexpr int smem = PrepSmem<T, DKT>::kBytes;
    static SmemLimit limit;
    cudaError_t e = limit.raise(k_delta_prep<T, DKT>, smem);
    if (e != cudaSuccess) return e;
    const long long units = slots(a.tokens, a.n) * a.hv;
    k_delta_prep<T, DKT><<<(unsigned)units, 256, smem, st>>>(a, (unsigned char *)ws,
                                                             (unsigned char *)ws + (size_t)units * kUnitBytes, flags);
    return cudaGetLastError();
}

template <typename T>
size_t bytes(long long slots, int hk, int hv, int dk) {
    return (size_t)slots * (hv * (size_t)kUnitBytes + hk * (size_t)(dk > 64 ? kq_bytes<T, 128>() : kq_bytes<T, 64>()));
}

}  // namespace

size_t delta_prep_bytes(int dtype, long long tokens, int n, int hk, int hv, int dk) {
    const long long c = slots(tokens, n);
    return dtype == S4_BF16 ? bytes<__nv_bfloat16>(c, hk, hv, dk)
                            : dtype == S4_F16 ? bytes<__half>(c, hk, hv, dk) : bytes<float>(c, hk, hv, dk);
}

cudaError_t launch_delta_prep(int dtype, const DeltaArgs &a, void *ws, unsigned *flags, cudaStream_t st) {
    const bool wide = a.dk > 64;
    if (dtype == S4_BF16)
        return wide ? run<__nv_bfloat16, 128>(a, ws, flags, st) : run<__nv_bfloat16, 64>(a, ws, flags, st);
    if (dtype == S4_F16) return wide ? run<__half, 128>(a, ws, flags, st) : run<__half, 64>(a, ws, flags, st);
    return wide ? run<float, 128>(a, ws, flags, st) : run<float, 64>(a, ws, flags, st);
}

}  // namespace s4
