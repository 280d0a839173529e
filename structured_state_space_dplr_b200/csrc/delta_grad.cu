// delta_grad.cu -- the chunked gated delta rule, backward within the chunks:
// the gradients of q, k, beta and g from the states before the chunks (S0),
// the state gradients behind them (dS1), E of the forward chain and dR of the
// backward chain. Per chunk and value head, with F = dO E^T, X = dR E^T,
// H_j = dS1 E_j and d_ij = e^(G_i - G_j):
//     M_ij = scale beta_j d_ij F_ij (j <= i),  N_ij = beta_j d_ij X_ij (j < i)
//     dq = scale e^G dO S0^T + M K
//     dk = -e^G dR S0^T + beta e^(G_C - G) H - (N + N^T) K + M^T Q
//     c1_j = sum_i scale d_ij q_i.k_j F_ij,  c2_j = sum_i d_ij k_i.k_j X_ij,
//     h_j = e^(G_C - G_j) k_j.H_j,   dbeta = c1 + h - c2
//     u_i = e^(G_i) (scale q_i.(S0 dO_i) - k_i.(S0 dR_i)),  W_ij the term of
//     beta_j (c1_j - c2_j) with row i,
//     dg_t = sum_{i >= t, j < t} W_ij + sum_{i >= t} u_i + sum_{j < t} beta_j h_j + e^(G_C) <S0, dS1>:
// what passes from before t to t or behind (the terms of the decay's sums on
// one side of t only cancel, and are left out).
//
// One block per chunk and key head, its value heads one after the other (their
// dq and dk are summed in registers, in order). Tensor-memory lane = row of the
// stacked [dR; dO], so dR's and dO's products share the instructions and the
// scalings of rows are scalings of threads. S0, dS1, E and dR are 192 KB in
// float at Dk = Dv = 128, read once and split into bf16 parts here. (As parts,
// stored by the chains and copied in bulk, they are half as much again, and
// <S0, dS1> then costs the backward chain more than the copies save.) That
// space allows one block per SM; what bounds it is the chain of conversions and
// products of a head. Measured: 4 x 4096 tokens, 16 key and 32
// value heads of 128 bf16 (4096 blocks) 1013 us, 1.9 GB read a time; tensor
// cores 28%, issue slots 28%, DRAM 22%. A head's E, dR and dO come to shared
// memory one head ahead, 1094 us without. Nine warps leave 168 registers a
// thread, of which heads of 128 spill: 380 bytes in bf16, 436 in half, 368 in
// float (a variable more alive throughout cost 1.5%).
#include "delta.cuh"
#include "s4dplr.h"

#include <type_traits>

namespace s4 {
namespace {

using namespace delta;

constexpr int kGradWarps = 8, kGradThreads = 32 * kGradWarps, kGradBlock = kGradThreads + 32;
constexpr int kTrLd = kC + 1;

// tensor-memory columns: the left operands' parts, X and F, [dR; dO] S0^T (later the sum of the last products), E dS1^T
constexpr int kTmA = 0, kTmXF = 192, kTmD = 256, kTmH = 384;

template <typename T, int DKT, int DVT>
struct GradSmem {
    static constexpr int kS = DVT * DKT * 2, kE = kC * DVT * 2, kKq = kq_bytes<T, DKT>();   // one part of S0 or dS1, of E; all of [K; Q]
    static constexpr int kSmall = 2 * kC * kTrLd * 4 + kC * 8 + 22 * kC * 4 + 128;
    // The states' image; before them a head's E, dR and dO as they are
    static constexpr int kRow = DVT * (int)sizeof(T) + 16;   // dO's rows, shifted banks
    static constexpr int kRaw = 2 * kC * DVT * 4 + kC * kRow, kFirst = 3 * kS > kRaw ? 3 * kS : kRaw;
    // [K; Q] stays beside it where there is room for both
    static constexpr bool kBeside = kFirst + 3 * kE + kKq + kSmall <= 232448;
    static constexpr int kArea = kBeside ? kFirst + kKq : (kFirst > kKq ? kFirst : kKq);
    static constexpr int kOffKq = kBeside ? kFirst : 0, kOffE = kArea, kOffSmall = kArea + 3 * kE;
    static constexpr int kBytes = kOffSmall + kSmall;
    static_assert(kBytes <= 232448, "shared memory of a block");
};

// 8 floats at p as three parts of 16 bytes, `part` bytes apart at dst
__device__ __forceinline__ void put_parts(unsigned char *dst, int part, const float (&f)[8]) {
    uint32_t w[4][3];
#pragma unroll
    for (int i = 0; i < 4; ++i) split<3>(f[2 * i], f[2 * i + 1], w[i]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
        *reinterpret_cast<uint4 *>(dst + q * part) = make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
}
// sums over the warp: lane l ends with the sum of the lanes' w[l] in w[0]
__device__ __forceinline__ void column_sums(float (&w)[32], int lane) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int t = 0; t < o; ++t) {
            const bool up = lane & o;
            const float other = __shfl_xor_sync(0xffffffffu, up ? w[t] : w[t + o], o);
            w[t] = (up ? w[t + o] : w[t]) + other;
        }
}

__device__ __forceinline__ void zero8(float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.0f;
}

// A state [dk / 4][dv][4] as right operand (rows v = K, columns dk): four pieces
// of 8 a thread at a time, the n0-th ones; first from memory, then as parts into
// the image. DOT: this thread's share of the dot with the state whose parts lie
// there so far (their sums are its floats to 24 bits).
template <int DKT, int DVT>
__device__ __forceinline__ void get_state(float (&f)[4][8], int n0, const float *u, int dk, int dv, int tid) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int n = (4 * n0 + k) * kGradThreads + tid, v = n & (DVT - 1), dg = n / DVT;
        zero8(f[k]);
        if (n < DVT * DKT / 8 && v < dv && 8 * dg < dk) {
            const float4 *q = reinterpret_cast<const float4 *>(u) + (size_t)2 * dg * dv + v;
            const float4 x = __ldg(q), y = __ldg(q + dv);
            f[k][0] = x.x, f[k][1] = x.y, f[k][2] = x.z, f[k][3] = x.w;
            f[k][4] = y.x, f[k][5] = y.y, f[k][6] = y.z, f[k][7] = y.w;
        }
    }
}
template <int DKT, int DVT, bool DOT>
__device__ __forceinline__ float put_state(unsigned char *dst, int part, const float (&f)[4][8], int n0, int tid) {
    float both = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int n = (4 * n0 + k) * kGradThreads + tid, v = n & (DVT - 1), dg = n / DVT;
        if (n >= DVT * DKT / 8) break;
        unsigned char *to = dst + (v >> 3) * 128 + dg * (DVT * 16) + (v & 7) * 16;
        if constexpr (DOT) {
            float z[8];
            zero8(z);
#pragma unroll
            for (int q = 2; q >= 0; --q) {
                const uint4 w = *reinterpret_cast<const uint4 *>(to + q * part);
                const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) z[2 * j] += lo_f(r[j]), z[2 * j + 1] += hi_f(r[j]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) both = fmaf(f[k][j], z[j], both);
        }
        put_parts(to, part, f[k]);
    }
    return both;
}

// 8 elements of shared memory, 16-byte aligned
__device__ __forceinline__ void take8(const float *p, float (&f)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void take8(const T *p, float (&f)[8]) {   // 16-bit types
    load_pack<T, 8>(p, f);
}

template <typename T, int DKT, int DVT>
__global__ void __launch_bounds__(kGradBlock, 1)
    k_delta_gradient(DeltaArgs a, const T *dout, const unsigned char *images, const float *keep_s, const float *keep_e,
                     const float *keep_ds, const float *keep_dr, T *dq, T *dk, float *dg, float *dbeta,
                     unsigned *flags) {
    using L = GradSmem<T, DKT, DVT>;
    constexpr int NB = Parts<T>::n, kPart = 2 * kC * DKT * 2, HK = DKT / 2, KV = DVT / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *kq = smem + L::kOffKq, *ei = smem + L::kOffE;
    float *tr = reinterpret_cast<float *>(smem + L::kOffSmall);              // N, M: [2][64][65]
    float2 *Gs = reinterpret_cast<float2 *>(tr + 2 * kC * kTrLd);
    float *bs = reinterpret_cast<float *>(Gs + kC);                          // beta
    float *eg = bs + kC, *dec = eg + kC;                                     // e^G, e^(G_C - G)
    float *ce = dec + kC, *de = ce + kC, *rf = de + kC;                      // factors of e^(G_i - G_j)
    float *csum = rf + kC;                                                   // [4][64]
    float *gsum = csum + 4 * kC, *rsum = gsum + 4 * kC;                      // [4][64], [128]
    float *dot = rsum + 2 * kC, *hdot = dot + 4 * kC;                        // [2][128], [2][64]
    float *red = hdot + 2 * kC;                                              // [8]
    uint64_t *bars = reinterpret_cast<uint64_t *>(red + 8);                  // kq, two products in flight, raw, end
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + 5);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int R = (warp & 3) * 32 + lane, i = R & (kC - 1), half = warp >> 2;   // row of [dR; dO] and of [K; Q], its token
    const bool low = R < kC;                                                    // a row of dR and K

    const long long slot = blockIdx.x / a.hk;
    const int hk = blockIdx.x % a.hk, per = a.hv / a.hk;
    const Chunk ch = chunk_of(a, slot);
    if (ch.rows <= 0) return;   // a slot no chunk uses
    const int rows = ch.rows;
    const long long tok = ch.tok;
    const long long orow = (long long)a.hv * a.dv;

    if (warp == 0) umma::tmem_alloc(tslot, 512);
    if (tid == 0) {
        for (int n = 0; n < 3; ++n) umma::mbar_init(bars + n, 1);
        umma::mbar_init(bars + 3, kGradThreads + 1);
        umma::mbar_init(bars + 4, 1);
        umma::fence_mbar_init();
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tm = uniform(*tslot);
    const uint32_t mine = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s0 = saddr(smem), kq0 = saddr(kq), e0 = saddr(ei);
    int kq_turn = 0, raw_loads = 0, turn1 = 0, turn2 = 0;
    bool ok = true;
    auto load_kq = [&]() {   // behind a barrier of the block; every thread waits
        if (ok && tid == 0) {
            mbar_expect(bars, L::kKq);
            bulk_load(kq, images + (size_t)(slot * a.hk + hk) * L::kKq, L::kKq, bars);
            mbar_arrive(bars);
        }
        try_wait(ok, bars, kq_turn++ & 1);
    };
    // operands written by these threads before, products (and bulk loads) behind;
    // a wait that ran out anywhere is known everywhere, and nothing more is issued
    auto barrier = [&]() {
        tm_wait_st();
        umma::fence_proxy_async();
        umma::fence_before_sync();
        ok = __syncthreads_and(ok);
        umma::fence_after_sync();
    };
    auto wait1 = [&]() {
        try_wait(ok, bars + 1, turn1++ & 1);
        umma::fence_after_sync();
    };
    auto wait2 = [&]() {
        try_wait(ok, bars + 2, turn2++ & 1);
        umma::fence_after_sync();
    };
    // D (+)= A [parts of K = 16 KS columns] times an image's PB parts
    auto times = [&](auto ks_n, auto pb, uint32_t d, uint32_t at, uint32_t lo, uint64_t b, uint32_t part, uint32_t step,
                     uint32_t id, bool first) {
#pragma unroll
        for (int o = 2; o >= 0; --o)
#pragma unroll
            for (int j = 0; j < decltype(pb)::value; ++j) {
                if (o - j < 0) continue;
                const int p = o - j;
#pragma unroll
                for (int ks = 0; ks < decltype(ks_n)::value; ++ks) {
                    mma_ts(tm + d, tm + (p < 2 ? at + 16 * ks + 8 * p : lo + 8 * ks),
                           b + ((j * part + ks * step) >> 4), id, !first);
                    first = false;
                }
            }
    };
    constexpr std::integral_constant<int, KV> kKv;
    constexpr std::integral_constant<int, kC / 16> kKc;
    constexpr std::integral_constant<int, 3> kThree;
    constexpr std::integral_constant<int, NB> kNb;
    if (warp == kGradWarps) {
        // the products, by a warp of their own: issuing them takes as long as they take
        load_kq();
        if (elect()) {
            bool acc = false;
#pragma unroll
            for (int o = 2; o >= 0; --o)
#pragma unroll
                for (int p = 0; p < NB; ++p) {
                    const int j = o - p;
                    if (j < 0 || j >= NB) continue;
#pragma unroll
                    for (int ks = 0; ks < DKT / 16; ++ks) {
                        umma::mma_bf16(tm + kTmXF, desc_k(kq0 + p * kPart + ks * 4096, 2048, 128),
                                       desc_k(kq0 + j * kPart + ks * 4096, 2048, 128), idesc(kC, false, false), acc);
                        acc = true;
                    }
                }
            umma::commit(bars + 1);
        }
        __syncwarp();
        // E and dR as they are to the place of the states' image, when nobody reads it
        auto load_raw = [&](int g) {
            if (elect() && ok) {
                ++raw_loads;
                const long long unit = slot * a.hv + hk * per + g;
                const uint32_t bytes = (uint32_t)(kC * a.dv) * 4;
                mbar_expect(bars + 3, 2 * bytes);
                bulk_load(smem, keep_e + (size_t)unit * kC * a.dv, bytes, bars + 3);
                bulk_load(smem + kC * DVT * 4, keep_dr + (size_t)unit * kC * a.dv, bytes, bars + 3);
                mbar_arrive(bars + 3);
            }
            __syncwarp();
        };
        if (L::kBeside) load_raw(0);
        for (int g = 0; g < per; ++g) {
            barrier();
            if (!ok) break;
            if (!L::kBeside) load_raw(g);
            barrier();
            if (elect()) {
                times(kKv, kThree, kTmXF, kTmA, kTmA + DVT, desc_k(e0, 1024, 128), L::kE, 2048, idesc(kC, false, false), true);
                umma::commit(bars + 1);
            }
            __syncwarp();
            barrier();
            if (elect()) {
                times(kKv, kThree, kTmD, kTmA, kTmA + DVT, desc_mn(s0, 128, DVT * 16), L::kS, 256, idesc(DKT, false, true),
                      true);
                umma::commit(bars + 2);
            }
            __syncwarp();
            barrier();
            if (elect()) {
                times(kKv, kThree, kTmH, kTmA, kTmA + DVT, desc_mn(s0, 128, DVT * 16), L::kS, 256, idesc(DKT, false, true),
                      true);
                umma::commit(bars + 1);
            }
            __syncwarp();
            if (L::kBeside && g + 1 < per) {
                try_wait(ok, bars + 1, 0);   // the phases' products: q.k, then X F and H in turn
                load_raw(g + 1);
            }
            if constexpr (!L::kBeside) {
                barrier();
                load_kq();
            }
            barrier();
            if (elect()) {
                times(kKc, kNb, kTmD, kTmA, kTmA + 64, desc_mn(kq0, 128, 2048), kPart, 256, idesc(DKT, false, true), true);
                times(kKc, kNb, kTmD, kTmA + 96, kTmA + 160, desc_mn(kq0 + 1024, 128, 2048), kPart, 256,
                      idesc(DKT, false, true), false);
                umma::commit(bars + 2);
            }
            __syncwarp();
            __syncthreads();
        }
        // the last products are done before the memory that they use goes, and the copies that nobody waits for any more
        if (elect()) umma::commit(bars + 4);
        __syncwarp();
        umma::mbar_wait(bars + 4, 0, kDrainLimit);
        if (!ok) drain_copies(bars + 3, raw_loads, 1);
    } else {
    // q_i.k_j and k_i.k_j, the same for all value heads
    load_kq();
    float raw[kC / 2];
    wait1();
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        float x[16];
        tm_ld16(mine + kTmXF + half * (kC / 2) + 16 * n, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) raw[16 * n + j] = x[j];
    }
    float acc[HK];   // this row of dk or dq, half of the columns
#pragma unroll
    for (int n = 0; n < HK; ++n) acc[n] = 0.0f;

    auto load_do = [&](int g) {   // dO's rows, padded, zeros behind the last
        if (!ok) return;
        constexpr int E = 16 / (int)sizeof(T), kPer = DVT / E;
        const T *src = dout + tok * orow + (long long)(hk * per + g) * a.dv;
        for (int n = tid; n < kC * kPer; n += kGradThreads) {
            const int r = n / kPer, c = n % kPer;
            const bool in = r < rows && c * E < a.dv;
            cp16(smem + 2 * kC * DVT * 4 + r * L::kRow + c * 16, in ? src + r * orow + c * E : dout, in);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(saddr(bars + 3)) : "memory");
    };
    if (L::kBeside) load_do(0);
    for (int g = 0; g < per; ++g) {
        const int hv = hk * per + g;
        const long long unit = slot * a.hv + hv;
        const float *us = keep_s + (size_t)unit * a.dk * a.dv, *ud = keep_ds + (size_t)unit * a.dk * a.dv;
        barrier();   // the last head's reads of shared and tensor memory
        if (!ok) break;
        if (!L::kBeside) load_do(g);
        if (warp == 1) {
            const GateSums gt = gate_sums(a, tok, hv, rows, lane);
            const int j = 2 * lane;
            const float xf = (float)gt.x, yf = (float)gt.y;
            Gs[j] = make_float2(xf, (float)(gt.x - xf));
            Gs[j + 1] = make_float2(yf, (float)(gt.y - yf));
            bs[j] = gt.b0;
            bs[j + 1] = gt.b1;
            const double all = __shfl_sync(0xffffffffu, gt.y, 31);
            eg[j] = exp2f(xf);
            eg[j + 1] = exp2f(yf);
            dec[j] = exp2f((float)(all - gt.x));
            dec[j + 1] = exp2f((float)(all - gt.y));
            // e^(G_i - G_j) as two factors: by G at the end of j's 16 tokens where i is behind them; within
            // the 16 by G of their first, while both factors are far from float's limits (2^60)
            const double end = __shfl_sync(0xffffffffu, gt.y, lane | 7), first = __shfl_sync(0xffffffffu, gt.x, lane & 24);
            const bool near = first - end < 60.0;
            ce[j] = exp2f((float)(end - gt.x));
            ce[j + 1] = exp2f((float)(end - gt.y));
            rf[j] = near ? exp2f((float)(gt.x - first)) : -1.0f;
            rf[j + 1] = near ? exp2f((float)(gt.y - first)) : -1.0f;
            de[j] = exp2f((float)(near ? first - gt.x : 0.0));
            de[j + 1] = exp2f((float)(near ? first - gt.y : 0.0));
        }
        float f[4][8];
        get_state<DKT, DVT>(f, 0, us, a.dk, a.dv, tid);   // on its way
        try_wait(ok, bars + 3, g & 1);
        // E as right operand (rows tokens, K = v)
#pragma unroll
        for (int u = 0; u < kC * DVT / 8 / kGradThreads; ++u) {
            const int n = u * kGradThreads + tid, t = n & (kC - 1), vg = n / kC;
            float e[8];
            zero8(e);
            if (8 * vg < a.dv) take8(reinterpret_cast<const float *>(smem) + (size_t)n * 8, e);
            put_parts(ei + (t >> 3) * 128 + vg * 1024 + (t & 7) * 16, L::kE, e);
        }
        // [dR; dO] as left operand, half of the columns a thread
#pragma unroll
        for (int n = 0; n < KV / 2; ++n) {
            const int ks = half * (KV / 2) + n;
            float x[16];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int v = 16 * ks + 8 * m;
                float y[8];
                zero8(y);
                if (low) {
                    if (v < a.dv) take8(reinterpret_cast<const float *>(smem + kC * DVT * 4) + ((v >> 3) * kC + i) * 8, y);
                } else {
                    take8(reinterpret_cast<const T *>(smem + 2 * kC * DVT * 4 + i * L::kRow) + v, y);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) x[8 * m + j] = y[j];
            }
            tm_split16(mine + kTmA + 16 * ks, mine + kTmA + DVT + 8 * ks, x);
        }
        barrier();
        // S0 as right operand, columns dk, K = v, beside the first product
        put_state<DKT, DVT, false>(smem, L::kS, f, 0, tid);
        if constexpr (DVT * DKT / 8 > 4 * kGradThreads) {
            get_state<DKT, DVT>(f, 1, us, a.dk, a.dv, tid);
            put_state<DKT, DVT, false>(smem, L::kS, f, 1, tid);
        }
        barrier();
        wait1();
        {   // N and M, to shared memory for their columns
            const float2 Gi = Gs[i];
            const float mul = low ? 1.0f : a.scale;
            float cw[kC / 2], pw[kC / 2], rs = 0.0f;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int j0 = half * (kC / 2) + 16 * n;
                if (j0 > (i | 31)) {   // above the diagonal for the whole warp
#pragma unroll
                    for (int t = 0; t < 16; ++t) cw[16 * n + t] = pw[16 * n + t] = tr[R * kTrLd + j0 + t] = 0.0f;
                    continue;
                }
                float x[16], e[16], be[16];
                get16(bs + j0, be);
                tm_ld16(mine + kTmXF + j0, x);
                if (j0 / 16 < i / 16) {
                    const float2 Gj = Gs[j0 + 15];
                    const float r = mul * exp2f((Gi.x - Gj.x) + (Gi.y - Gj.y));
                    get16(ce + j0, e);
#pragma unroll
                    for (int t = 0; t < 16; ++t) x[t] *= r * e[t];
                } else if (j0 / 16 == i / 16) {
                    const int m = low ? i : i + 1;
                    const float r = rf[i];
                    if (r >= 0.0f) {   // the same for the 16 tokens
                        get16(de + j0, e);
#pragma unroll
                        for (int t = 0; t < 16; ++t) x[t] = j0 + t < m ? x[t] * (mul * r * e[t]) : 0.0f;
                    } else {
#pragma unroll
                        for (int t = 0; t < 16; ++t) {
                            const float2 Gj = Gs[j0 + t];
                            x[t] = j0 + t < m ? x[t] * mul * exp2f((Gi.x - Gj.x) + (Gi.y - Gj.y)) : 0.0f;
                        }
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < 16; ++t) x[t] = 0.0f;
                }
#pragma unroll
                for (int t = 0; t < 16; ++t) {
                    cw[16 * n + t] = x[t] * raw[16 * n + t];
                    pw[16 * n + t] = j0 + t <= i ? rs : 0.0f;   // what this half's columns before j hand to row i >= j
                    rs = fmaf(be[t], cw[16 * n + t], rs);
                    tr[R * kTrLd + j0 + t] = be[t] * x[t];
                }
            }
            if (half == 0) rsum[R] = rs;
            if (half * (kC / 2) <= (i | 31)) {   // else zeros
                column_sums(cw, lane);
                column_sums(pw, lane);
            }
            csum[(warp & 3) * kC + half * (kC / 2) + lane] = cw[0];
            gsum[(warp & 3) * kC + half * (kC / 2) + lane] = pw[0];
        }
        get_state<DKT, DVT>(f, 0, ud, a.dk, a.dv, tid);
        wait2();   // the left operand and S0 are used up
        if (low) {   // E as left operand (rows 64-127 of the product go unread)
#pragma unroll
            for (int n = 0; n < KV / 2; ++n) {
                const int ks = half * (KV / 2) + n;
                const unsigned char *src = ei + (i >> 3) * 128 + 2 * ks * 1024 + (i & 7) * 16;
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(src + p * L::kE);
                    const uint4 w = *reinterpret_cast<const uint4 *>(src + p * L::kE + 1024);
                    const uint32_t r[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
                    tm_st8(mine + kTmA + (p < 2 ? 16 * ks + 8 * p : DVT + 8 * ks), r);
                }
            }
        }
        float both = put_state<DKT, DVT, true>(smem, L::kS, f, 0, tid);   // <S0, dS1>
        if constexpr (DVT * DKT / 8 > 4 * kGradThreads) {
            get_state<DKT, DVT>(f, 1, ud, a.dk, a.dv, tid);
            both += put_state<DKT, DVT, true>(smem, L::kS, f, 1, tid);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) both += __shfl_xor_sync(0xffffffffu, both, o);
        if (lane == 0) red[warp] = both;
        barrier();
        // a product with a state, into dk or dq and its dot with k or q
        auto take = [&](uint32_t at, float scale) {
            float d0 = 0.0f;
#pragma unroll
            for (int n = 0; n < HK; n += 16) {
                const int d = half * HK + n;
                float x[16], k[16];
                tm_ld16(mine + at + d, x);
                const unsigned char *src = kq + (R >> 3) * 128 + (d >> 3) * 2048 + (R & 7) * 16;
#pragma unroll
                for (int t = 0; t < 16; ++t) k[t] = 0.0f;
#pragma unroll
                for (int p = NB - 1; p >= 0; --p)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(src + p * kPart + q * 2048);
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            k[8 * q + 2 * t] += lo_f(w[t]);
                            k[8 * q + 2 * t + 1] += hi_f(w[t]);
                        }
                    }
#pragma unroll
                for (int t = 0; t < 16; ++t) {
                    d0 = fmaf(x[t], k[t], d0);
                    acc[n + t] = fmaf(scale, x[t], acc[n + t]);
                }
            }
            return d0;
        };
        // -e^G k.(S0 dR); scale e^G q.(S0 dO)
        const float sr = low ? -eg[i] : a.scale * eg[i];
        if constexpr (L::kBeside) dot[half * 2 * kC + R] = sr * take(kTmD, sr);   // beside the product
        wait1();
        if (L::kBeside && g + 1 < per) load_do(g + 1);
        if constexpr (!L::kBeside) {
            barrier();
            load_kq();
            dot[half * 2 * kC + R] = sr * take(kTmD, sr);
        }
        // left operands of the products with K (-(N + N^T); M) and Q (M^T; 0)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int j0 = half * (kC / 2) + 16 * n;
            float x[16], y[16];
#pragma unroll
            for (int t = 0; t < 16; ++t) {
                const int j = j0 + t;
                x[t] = low ? -(tr[i * kTrLd + j] + tr[j * kTrLd + i]) : tr[R * kTrLd + j];
                y[t] = low ? tr[(kC + j) * kTrLd + i] : 0.0f;
            }
            tm_split16(mine + kTmA + j0, mine + kTmA + 64 + j0 / 2, x);
            tm_split16(mine + kTmA + 96 + j0, mine + kTmA + 160 + j0 / 2, y);
        }
        barrier();
        if (low) {   // H, beside the last products (warps 0, 1, 4 and 5)
            const float d1 = take(kTmH, bs[i] * dec[i]);
            hdot[half * kC + i] = dec[i] * d1;
        }
        __syncthreads();
        if (warp == 1) {   // dbeta and dg, two tokens a lane
            float rect[2], u[2], r0[2], bh[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int j = 2 * lane + t;
                const float c2 = csum[j] + csum[kC + j], c1 = csum[2 * kC + j] + csum[3 * kC + j];
                const float hj = hdot[j] + hdot[kC + j];
                if (j < rows) dbeta[(tok + j) * a.hv + hv] = (c1 - c2) + hj;
                bh[t] = bs[j] * hj;
                rect[t] = (gsum[2 * kC + j] + gsum[3 * kC + j]) - (gsum[j] + gsum[kC + j]);
                u[t] = (dot[j] + dot[2 * kC + j]) + (dot[kC + j] + dot[3 * kC + j]);
                r0[t] = rsum[kC + j] - rsum[j];   // of the first 32 columns: for t >= 32 they are all before t
            }
            float ss = 0.0f;
#pragma unroll
            for (int w = 0; w < kGradWarps; ++w) ss += red[w];
            // from this lane's first token on; before it
            float su = u[0] + u[1], sr = r0[0] + r0[1], sb = bh[0] + bh[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float z0 = __shfl_down_sync(0xffffffffu, su, o), z1 = __shfl_down_sync(0xffffffffu, sr, o);
                const float z2 = __shfl_up_sync(0xffffffffu, sb, o);
                if (lane + o < 32) su += z0, sr += z1;
                if (lane >= o) sb += z2;
            }
            sb = __shfl_up_sync(0xffffffffu, sb, 1);
            if (lane == 0) sb = 0.0f;
            const float all = eg[kC - 1] * ss;
            const int j = 2 * lane;
            const bool late = lane >= 16;
            if (j < rows) dg[(tok + j) * a.hv + hv] = (rect[0] + (late ? sr : 0.0f)) + su + sb + all;
            if (j + 1 < rows)
                dg[(tok + j + 1) * a.hv + hv] =
                    (rect[1] + (late ? sr - r0[0] : 0.0f)) + (su - u[0]) + (sb + bh[0]) + all;
        }
        wait2();
#pragma unroll
        for (int n = 0; n < HK; n += 16) {
            float x[16];
            tm_ld16(mine + kTmD + half * HK + n, x);
#pragma unroll
            for (int t = 0; t < 16; ++t) acc[n + t] += x[t];
        }
    }
    if (!ok) drain_copies(bars, tid == 0 ? kq_turn : 0, 1);   // (a load left out is waited for in vain, to the limit)
    if (i < rows) {
        T *o = (low ? dk : dq) + ((tok + i) * a.hk + hk) * a.dk + half * HK;
#pragma unroll
        for (int n = 0; n < HK; n += 8)
            if (half * HK + n < a.dk) {
                const float f[8] = {acc[n],     acc[n + 1], acc[n + 2], acc[n + 3],
                                    acc[n + 4], acc[n + 5], acc[n + 6], acc[n + 7]};
                if constexpr (sizeof(T) == 2) {
                    store_pack<T, 8>(o + n, f);
                } else {
                    *reinterpret_cast<float4 *>(o + n) = make_float4(f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<float4 *>(o + n + 4) = make_float4(f[4], f[5], f[6], f[7]);
                }
            }
    }
    }
    if (!ok && flags) atomicOr(flags, S4_FLAG_TIMEOUT);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    if (warp == 0) umma::tmem_dealloc(tm, 512);
}

template <typename T, int DKT, int DVT>
cudaError_t run(const DeltaArgs &a, const void *dout, const void *ws, const float *keep_s, const float *keep_e,
                const float *keep_ds, const float *keep_dr, void *dq, void *dk, float *dg, float *dbeta,
                unsigned *flags, cudaStream_t st) {
    constexpr int smem = GradSmem<T, DKT, DVT>::kBytes;
    static SmemLimit limit;
    cudaError_t e = limit.raise(k_delta_gradient<T, DKT, DVT>, smem);
    if (e != cudaSuccess) return e;
    const long long n = slots(a.tokens, a.n);
    k_delta_gradient<T, DKT, DVT><<<(unsigned)(n * a.hk), kGradBlock, smem, st>>>(
        a, (const T *)dout, (const unsigned char *)ws + (size_t)n * a.hv * kUnitBytes, keep_s, keep_e, keep_ds, keep_dr,
        (T *)dq, (T *)dk, dg, dbeta, flags);
    return cudaGetLastError();
}

template <typename T, typename... Args>
cudaError_t by_size(const DeltaArgs &a, Args... args) {
    if (a.dk > 64) return a.dv > 64 ? run<T, 128, 128>(a, args...) : run<T, 128, 64>(a, args...);
    return a.dv > 64 ? run<T, 64, 128>(a, args...) : run<T, 64, 64>(a, args...);
}

}  // namespace

cudaError_t launch_delta_gradient(int dtype, const DeltaArgs &a, const void *dout, const void *ws, const float *keep_s,
                                  const float *keep_e, const float *keep_ds, const float *keep_dr, void *dq, void *dk,
                                  float *dg, float *dbeta, unsigned *flags, cudaStream_t st) {
    if (dtype == S4_BF16)
        return by_size<__nv_bfloat16>(a, dout, ws, keep_s, keep_e, keep_ds, keep_dr, dq, dk, dg, dbeta, flags, st);
    if (dtype == S4_F16)
        return by_size<__half>(a, dout, ws, keep_s, keep_e, keep_ds, keep_dr, dq, dk, dg, dbeta, flags, st);
    return by_size<float>(a, dout, ws, keep_s, keep_e, keep_ds, keep_dr, dq, dk, dg, dbeta, flags, st);
}

}  // namespace s4
