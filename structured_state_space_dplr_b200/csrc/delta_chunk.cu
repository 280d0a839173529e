// delta_chunk.cu -- the chunked gated delta rule, forward: one block walks the
// chunks of one sequence and value head with the state in registers.
//
// Everything is kept transposed, value channel = tensor-memory lane, so that
// the three products of a chunk that depend on each other take their left
// operand from tensor memory, written there by the threads that computed it,
// and their right operand from the natural image of K, Q or [T; PT]:
//     D1 = S0^T [K; Q]^T          (128 x 64 each)
//     R^T = V^T - e^G D1k  ->  D2 = R^T [T; PT]^T  = [E^T | (PT R)^T]
//     (beta e^(G_C - G) E)^T  ->  D3 = (..)^T K     (128 x Dk)
//     S1^T = e^(G_C) S0^T + D3,   O^T = scale e^G D1q + D2o.
// Roles: warps 0-7 the element-wise steps (two warps per lane quarter, each
// half the columns), warp 8 issues the products, warps 9-11 load.
//
// What bounds it: the chain of a chunk, three products and three passes of
// splitting and tensor-memory traffic, one after the other; the products that
// are not in the chain (D1q, D2o) and the output run beside it. A block needs
// all 512 tensor-memory columns, so there is one per SM.
#include "delta.cuh"
#include "s4dplr.h"

namespace s4 {
namespace {

using namespace delta;

constexpr int kEpiWarps = 8, kLoadWarps = 3, kThreads = (kEpiWarps + 1 + kLoadWarps) * 32;

// tensor-memory columns: the state's parts (and D3 in their place), the parts
// of R (in the place of D1k) and of beta e^(G_C - G) E (in the place of D2e),
// D1q, D2o. A warp overwrites only columns that it alone has read: half h of
// the K range holds its high and middle parts in the accumulator columns of
// the same half.
constexpr int kTmS = 0, kTmR = 192, kTmE = 288, kTmQ = 384, kTmO = 448;

// column of part p, K step ks (8 columns of 16 elements), in an operand of K
// elements that lies in the place of an accumulator of K columns
template <int K>
__device__ __forceinline__ uint32_t part_col(int p, int ks) {
    constexpr int half = K / 2;
    const int h = ks / (half / 16), r = ks % (half / 16);
    return p < 2 ? h * half + p * (half / 2) + 8 * r : K + h * (half / 2) + 8 * r;
}

template <typename T, int DKT>
struct ChainSmem {
    static constexpr int kImg = kC * DKT * 2;                                    // one part of K or Q
    static constexpr int kStage = 2 * Parts<T>::n * kImg + kUnitBytes;           // K, Q, [T; PT], factors
    static constexpr int kBars = 256;
    static constexpr int kStages = 2 * kStage + kBars <= 232448 ? 2 : 1;
    static constexpr int kBytes = kStages * kStage + kBars;
    static_assert(kBytes <= 232448, "shared memory of a block");
};

enum { bFull = 0, bEmpty = 2, bS = 4, bR, bE, bO, bM1, bM2, bM2o, bM3, bCount };

template <typename T, int DKT>
__global__ void __launch_bounds__(kThreads, 1) k_delta_forward(DeltaArgs a, const float *init, float *last,
                                                               const unsigned char *ws, float *keep_s, float *keep_e,
                                                               unsigned *flags) {
    using L = ChainSmem<T, DKT>;
    constexpr int NB = Parts<T>::n, ST = L::kStages, HC = DKT / 2;
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + ST * L::kStage);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + bCount);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hv = blockIdx.x % a.hv, s = blockIdx.x / a.hv, hk = hv / (a.hv / a.hk);
    const Seq sq = sequence(a, s);
    const int chunks = (sq.len + kC - 1) / kC;

    if (warp == 0) umma::tmem_alloc(tslot, 512);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(bars + bFull + i, kLoadWarps * 32 + 1);
            umma::mbar_init(bars + bEmpty + i, 1 + kEpiWarps);
        }
        for (int i = bS; i <= bO; ++i) umma::mbar_init(bars + i, kEpiWarps);
        for (int i = bM1; i <= bM3; ++i) umma::mbar_init(bars + i, 1);
        umma::fence_mbar_init();
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tm = *tslot;
    bool ok = true;

    if (warp >= kEpiWarps + 1) {
        // ------------------------------------------------------ loading ----
        const int w = warp - kEpiWarps - 1, lt = w * 32 + lane;
        for (int c = 0; c < chunks && ok; ++c) {
            const int st = c % ST, turn = c / ST;
            unsigned char *sp = smem + st * L::kStage;
            const long long tok = sq.tok0 + (long long)c * kC;
            const int rows = sq.len - c * kC < kC ? sq.len - c * kC : kC;
            constexpr int kUnits = 2 * (kC / 8) * (DKT / 32), kBatch = 4;   // K then Q; 8 rows x 4 column groups
            // the next chunk's V on its way to L2: the element-wise warps read it from there
            for (int r = lt; r < kC; r += kLoadWarps * 32)
                if (c * kC + kC + r < sq.len) {
                    const char *p = (const char *)((const T *)a.v + (tok + kC + r) * a.sv + (long long)hv * a.dv);
                    for (int b = 0; b < a.dv * (int)sizeof(T); b += 128)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(p + b));
                }
            bool waited = false;
            for (int u0 = w; u0 < kUnits; u0 += kLoadWarps * kBatch) {
                uint4 p[kBatch][NB];
#pragma unroll
                for (int n = 0; n < kBatch; ++n) {
                    const int u = u0 + n * kLoadWarps;
                    const int row = (u / (DKT / 32)) % (kC / 8) * 8 + (lane & 7), cg = (u % (DKT / 32)) * 4 + (lane >> 3);
#pragma unroll
                    for (int i = 0; i < NB; ++i) p[n][i] = make_uint4(0, 0, 0, 0);
                    if (u < kUnits && row < rows && 8 * cg < a.dk) {
                        const T *src = u < kUnits / 2 ? (const T *)a.k + (tok + row) * a.sk
                                                      : (const T *)a.q + (tok + row) * a.sq;
                        load_parts(src + (long long)hk * a.dk + 8 * cg, p[n]);
                    }
                }
                if (!waited) {   // the stage is free (its first use needs no wait)
                    waited = true;
                    ok = umma::mbar_wait(bars + bEmpty + st, (turn & 1) ^ 1, kSpinLimit);
                    if (!ok) break;
                    if (lt == 0) {
                        mbar_expect(bars + bFull + st, kUnitBytes);
                        bulk_load(sp + 2 * NB * L::kImg,
                                  ws + (size_t)((sq.slot0 + c) * a.hv + hv) * kUnitBytes, kUnitBytes,
                                  bars + bFull + st);
                    }
                }
#pragma unroll
                for (int n = 0; n < kBatch; ++n) {
                    const int u = u0 + n * kLoadWarps;
                    if (u >= kUnits) break;
                    const int row = (u / (DKT / 32)) % (kC / 8) * 8 + (lane & 7), cg = (u % (DKT / 32)) * 4 + (lane >> 3);
#pragma unroll
                    for (int i = 0; i < NB; ++i)
                        *reinterpret_cast<uint4 *>(sp + ((u < kUnits / 2 ? 0 : NB) + i) * L::kImg + (row >> 3) * 128 +
                                                   cg * 1024 + (row & 7) * 16) = p[n][i];
                }
            }
            if (!ok) break;
            umma::fence_proxy_async();
            mbar_arrive(bars + bFull + st);
        }
        // every copy has been waited for by the readers, unless a wait ran out: then here
        if (!ok && lt == 0)
            for (int i = 0; i < ST; ++i) umma::mbar_wait(bars + bFull + i, 0, 1u << 16);
    } else if (warp == kEpiWarps) {
        // ----------------------------------------------------- products ----
        for (int c = 0; c < chunks && ok; ++c) {
            const int st = c % ST, par = (c / ST) & 1, pc = c & 1;
            const uint32_t k0 = saddr(smem + st * L::kStage), q0 = k0 + NB * L::kImg, t0 = k0 + 2 * NB * L::kImg;
            ok = umma::mbar_wait(bars + bFull + st, par, kSpinLimit) && umma::mbar_wait(bars + bS, pc, kSpinLimit) &&
                 (c == 0 || umma::mbar_wait(bars + bM2o, pc ^ 1, kSpinLimit));   // R's parts have been read
            if (!ok) break;
            umma::fence_after_sync();
            auto state_times = [&](uint32_t d, uint32_t img) {   // D = S0^T (K or Q)^T
                bool acc = false;
#pragma unroll
                for (int o = 2; o >= 0; --o)
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        if (o - j < 0) continue;
#pragma unroll
                        for (int ks = 0; ks < DKT / 16; ++ks) {
                            mma_ts(tm + d, tm + kTmS + part_col<DKT>(o - j, ks),
                                   desc_k(img + j * L::kImg + ks * 2048, 1024, 128), idesc(kC, false, false), acc);
                            acc = true;
                        }
                    }
            };
            // D = R^T T^T or R^T PT^T (rows from `row0`); both are lower
            // triangular, so K step ks meets rows 16 ks and up only
            auto r_times = [&](uint32_t d, int row0) {
                bool acc = false;
#pragma unroll
                for (int o = 2; o >= 0; --o)
#pragma unroll
                    for (int j = 0; j <= o; ++j)
#pragma unroll
                        for (int ks = 0; ks < kC / 16; ++ks) {
                            mma_ts(tm + d + 16 * ks, tm + kTmR + part_col<kC>(o - j, ks),
                                   desc_k(t0 + j * kTpImage + ks * 4096 + (row0 / 8 + 2 * ks) * 128, 2048, 128),
                                   idesc(kC - 16 * ks, false, false), acc || ks > 0);
                            if (ks == kC / 16 - 1) acc = true;
                        }
            };
            if (lane == 0) {
                state_times(kTmR, k0);
                umma::commit(bars + bM1);
            }
            __syncwarp();
            // D1q and D2o of the chunk before have been read
            ok = c == 0 || umma::mbar_wait(bars + bO, pc ^ 1, kSpinLimit);
            if (!ok) break;
            umma::fence_after_sync();
            if (lane == 0) state_times(kTmQ, q0);
            __syncwarp();
            ok = umma::mbar_wait(bars + bR, pc, kSpinLimit);
            if (!ok) break;
            umma::fence_after_sync();
            if (lane == 0) {
                r_times(kTmE, 0);
                umma::commit(bars + bM2);
            }
            __syncwarp();
            ok = umma::mbar_wait(bars + bE, pc, kSpinLimit);
            if (!ok) break;
            umma::fence_after_sync();
            if (lane == 0) {   // D3 = (beta e^(G_C - G) E)^T K, in the place of the state's parts
                bool acc = false;
#pragma unroll
                for (int o = 2; o >= 0; --o)
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        if (o - j < 0) continue;
#pragma unroll
                        for (int ks = 0; ks < kC / 16; ++ks) {
                            mma_ts(tm + kTmS, tm + kTmE + part_col<kC>(o - j, ks),
                                   desc_mn(k0 + j * L::kImg + ks * 256, 128, 1024), idesc(DKT, false, true), acc);
                            acc = true;
                        }
                    }
                umma::commit(bars + bM3);
                r_times(kTmO, kC);
                umma::commit(bars + bM2o);
                umma::commit(bars + bEmpty + st);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------- element-wise ----
        const int h = warp >> 2, v = (warp & 3) * 32 + lane;   // half of the columns, value channel
        const uint32_t mine = tm + ((uint32_t)((warp & 3) * 32) << 16);
        const bool vin = v < a.dv;
        float S[HC];
        const size_t st0 = ((size_t)s * a.hv + hv) * a.dk * a.dv + v;
#pragma unroll
        for (int i = 0; i < HC; ++i) {
            const int d = h * HC + i;
            S[i] = init && vin && d < a.dk ? __ldg(init + st0 + (size_t)d * a.dv) : 0.0f;
        }
        auto put_state = [&]() {
#pragma unroll
            for (int i = 0; i < HC; i += 16) {
                float x[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = S[i + j];
                tm_split16(mine + kTmS + part_col<DKT>(0, (h * HC + i) / 16),
                           mine + kTmS + part_col<DKT>(1, (h * HC + i) / 16),
                           mine + kTmS + part_col<DKT>(2, (h * HC + i) / 16), x);
            }
            tm_wait_st();
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + bS);
        };
        auto put_output = [&](int c) {   // O of chunk c, once PT R has arrived
            const int st = c % ST;
            const float *eg = reinterpret_cast<const float *>(smem + st * L::kStage + 2 * NB * L::kImg + kTpBytes);
            ok = umma::mbar_wait(bars + bM2o, c & 1, kSpinLimit) && ok;
            umma::fence_after_sync();
#pragma unroll
            for (int i = 0; i < kC / 2; i += 16) {
                const int j0 = h * (kC / 2) + i;
                float x[16], y[16];
                tm_ld16(mine + kTmQ + j0, x);
                tm_ld16(mine + kTmO + j0, y);
                T *o = (T *)a.o + ((sq.tok0 + (long long)c * kC + j0) * a.hv + hv) * a.dv + v;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (vin && c * kC + j0 + j < sq.len)
                        o[(size_t)j * a.hv * a.dv] = from_f<T>(fmaf(a.scale * eg[j0 + j], x[j], y[j]));
            }
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bars + bO);
                mbar_arrive(bars + bEmpty + st);
            }
        };
        if (chunks) put_state();
        for (int c = 0; c < chunks && ok; ++c) {
            const int st = c % ST, pc = c & 1;
            const float *eg = reinterpret_cast<const float *>(smem + st * L::kStage + 2 * NB * L::kImg + kTpBytes);
            const long long unit = (sq.slot0 + c) * a.hv + hv;
            T vr[kC / 2];   // V^T of this thread's tokens, on its way while the output is written
            {
                const T *vp = (const T *)a.v + (sq.tok0 + (long long)c * kC + h * (kC / 2)) * a.sv +
                              (long long)hv * a.dv + v;
#pragma unroll
                for (int j = 0; j < kC / 2; ++j)
                    vr[j] = vin && c * kC + h * (kC / 2) + j < sq.len ? vp[(long long)j * a.sv] : from_f<T>(0.0f);
            }
            if (keep_s && vin) {   // the state before the chunk
                float *ks = keep_s + (size_t)unit * a.dk * a.dv + v;
#pragma unroll
                for (int i = 0; i < HC; ++i)
                    if (h * HC + i < a.dk) ks[(size_t)(h * HC + i) * a.dv] = S[i];
            }
            if (c > 0) put_output(c - 1);
            ok = ok && umma::mbar_wait(bars + bFull + st, (c / ST) & 1, kSpinLimit) &&
                 umma::mbar_wait(bars + bM1, pc, kSpinLimit);
            if (!ok) break;
            umma::fence_after_sync();
#pragma unroll
            for (int i = 0; i < kC / 2; i += 16) {   // R^T = V^T - e^G D1k
                const int j0 = h * (kC / 2) + i;
                float x[16];
                tm_ld16(mine + kTmR + j0, x);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = fmaf(-eg[j0 + j], x[j], to_f(vr[i + j]));
                // the parts go where this half's accumulators were: both groups are read before either is written
                if (i == 0) {
                    float y[16];
                    tm_ld16(mine + kTmR + j0 + 16, y);
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = fmaf(-eg[j0 + 16 + j], y[j], to_f(vr[16 + j]));
                    tm_split16(mine + kTmR + part_col<kC>(0, j0 / 16), mine + kTmR + part_col<kC>(1, j0 / 16),
                               mine + kTmR + part_col<kC>(2, j0 / 16), x);
                    tm_split16(mine + kTmR + part_col<kC>(0, j0 / 16 + 1), mine + kTmR + part_col<kC>(1, j0 / 16 + 1),
                               mine + kTmR + part_col<kC>(2, j0 / 16 + 1), y);
                    break;
                }
            }
            tm_wait_st();
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + bR);
            ok = umma::mbar_wait(bars + bM2, pc, kSpinLimit);
            if (!ok) break;
            umma::fence_after_sync();
            {   // E^T, and beta e^(G_C - G) E as the next operand
                const int j0 = h * (kC / 2);
                float x[16], y[16];
                tm_ld16(mine + kTmE + j0, x);
                tm_ld16(mine + kTmE + j0 + 16, y);
                if (keep_e && vin) {
                    float *ke = keep_e + ((size_t)unit * kC + j0) * a.dv + v;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        ke[(size_t)j * a.dv] = x[j];
                        ke[(size_t)(j + 16) * a.dv] = y[j];
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    x[j] *= eg[kC + j0 + j];
                    y[j] *= eg[kC + j0 + 16 + j];
                }
                tm_split16(mine + kTmE + part_col<kC>(0, j0 / 16), mine + kTmE + part_col<kC>(1, j0 / 16),
                           mine + kTmE + part_col<kC>(2, j0 / 16), x);
                tm_split16(mine + kTmE + part_col<kC>(0, j0 / 16 + 1), mine + kTmE + part_col<kC>(1, j0 / 16 + 1),
                           mine + kTmE + part_col<kC>(2, j0 / 16 + 1), y);
            }
            tm_wait_st();
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + bE);
            ok = umma::mbar_wait(bars + bM3, pc, kSpinLimit);
            if (!ok) break;
            umma::fence_after_sync();
            const float total = eg[kC - 1];   // e^(G_C): rows past the end have g = 0
#pragma unroll
            for (int i = 0; i < HC; i += 16) {
                float x[16];
                tm_ld16(mine + kTmS + h * HC + i, x);
#pragma unroll
                for (int j = 0; j < 16; ++j) S[i + j] = fmaf(total, S[i + j], x[j]);
            }
            if (c + 1 < chunks) put_state();
        }
        if (ok && chunks) put_output(chunks - 1);
        if (last && vin) {
#pragma unroll
            for (int i = 0; i < HC; ++i)
                if (h * HC + i < a.dk) last[st0 + (size_t)(h * HC + i) * a.dv] = S[i];
        }
    }
    if (!ok && flags && lane == 0) atomicOr(flags, S4_FLAG_TIMEOUT);
    // a wait that ran out may leave products in flight
    if (warp == kEpiWarps && !ok) {
        if (lane == 0) umma::commit(bars + bM3);
        __syncwarp();
        umma::mbar_wait(bars + bM3, 0, 1u << 16);
        umma::mbar_wait(bars + bM3, 1, 1u << 16);
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    if (warp == 0) umma::tmem_dealloc(tm, 512);
}

template <typename T, int DKT>
cudaError_t run(const DeltaArgs &a, const float *init, float *last, const void *ws, float *keep_s, float *keep_e,
                unsigned *flags, cudaStream_t st) {
    constexpr int smem = ChainSmem<T, DKT>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(k_delta_forward<T, DKT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    k_delta_forward<T, DKT><<<a.n * a.hv, kThreads, smem, st>>>(a, init, last, (const unsigned char *)ws, keep_s,
                                                                keep_e, flags);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_forward(int dtype, const DeltaArgs &a, const float *init, float *last, const void *ws,
                                 float *keep_s, float *keep_e, unsigned *flags, cudaStream_t st) {
    const bool wide = a.dk > 64;
    if (dtype == S4_BF16)
        return wide ? run<__nv_bfloat16, 128>(a, init, last, ws, keep_s, keep_e, flags, st)
                    : run<__nv_bfloat16, 64>(a, init, last, ws, keep_s, keep_e, flags, st);
    if (dtype == S4_F16)
        return wide ? run<__half, 128>(a, init, last, ws, keep_s, keep_e, flags, st)
                    : run<__half, 64>(a, init, last, ws, keep_s, keep_e, flags, st);
    return wide ? run<float, 128>(a, init, last, ws, keep_s, keep_e, flags, st)
                : run<float, 64>(a, init, last, ws, keep_s, keep_e, flags, st);
}

}  // namespace s4
