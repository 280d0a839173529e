// delta_back.cu -- the chunked gated delta rule, backward in the states: one
// block walks the chunks of one sequence and value head from the last to the
// first with the state's gradient in registers.
//
// With dS1 the gradient of the state behind a chunk (transposed like the
// forward chain, value channel = tensor-memory lane):
//     D1 = dS1^T K^T                                         (128 x 64)
//     dR^T = (beta e^(G_C - G) D1) T + dO^T PT               (128 x 64)
//     dS0^T = e^(G_C) dS1^T + (scale e^G dO)^T Q - (e^G dR)^T K   (128 x Dk)
// dR is the gradient of V and, with dS1, what the gradient kernel needs. The
// products with dO do not depend on the chain and fill its gaps. T and PT are
// read by columns (MN-major) from the forward's images, 16 columns a product.
// Roles and bounds as in the forward chain. Measured: 4 x 4096 tokens, 32 heads
// of 128 bf16 337 us, 5.3 us a chunk.
#include "delta.cuh"
#include "s4dplr.h"

namespace s4 {
namespace {

using namespace delta;

// Tensor-memory columns; parts in the place of the accumulator they come from
// (16 columns by 16 columns), their low ones apart:
//   kTmS   the state gradient's parts (128), D3 in their place, low kTmSl
//   kTmK   dS1^T K^T (64), then the parts of its scaled value, low kTmKl
//   kTmR   dR^T (64), then the parts of -e^G dR, low kTmRl
//   kTmX   the parts of dO (64 columns), low kTmXl; later those of scale e^G dO
constexpr int kTmS = 0, kTmSl = 128, kTmK = 192, kTmR = 256, kTmX = 320, kTmKl = 384, kTmRl = 416, kTmXl = 448;

enum { bFull = 0, bEmpty = 2, bS = 4, bK = 8, bR = 10, bX = 12, bY, bM1, bMx, bM2, bM3, bEnd, bCount };

// SUM: dN of a segment, the state's gradient before it from none behind it,
// without output. Otherwise the segment itself, from the gradient behind it.
template <typename T, int DKT, bool SUM>
__global__ void __launch_bounds__(kThreads, 1) k_delta_backward(DeltaArgs a, const T *dout, const float *dlast,
                                                                float *dinit, float *sums, const unsigned char *ws,
                                                                const unsigned char *images, T *dv, float *keep_ds,
                                                                float *keep_dr, unsigned *flags) {
    using L = Stage<T, DKT>;
    constexpr int NB = Parts<T>::n, HC = DKT / 2, NS = DKT / 32;   // NS: K steps of a half of the state
    extern __shared__ __align__(1024) unsigned char smem[];
    const int ST = L::count(a.dv), stage_bytes = L::bytes(a.dv);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + ST * stage_bytes);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + bCount);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int hv = blockIdx.x % a.hv, hk = hv / (a.hv / a.hk);
    const Segment sg = segment_of(a, blockIdx.x / a.hv);
    if (sg.s < 0 || (SUM && sg.index == 0)) return;
    const Summaries su(a.dk, a.dv, true);
    Seq sq = sequence(a, sg.s);   // from here on the segment as a sequence
    sq.tok0 += (long long)sg.first * kC;
    sq.slot0 += sg.first;
    sq.len = sq.len - sg.first * kC < sg.chunks * kC ? sq.len - sg.first * kC : sg.chunks * kC;
    const int chunks = uniform(sg.chunks);
    const long long orow = (long long)a.hv * a.dv;   // dO and dV are contiguous

    if (warp == 0) umma::tmem_alloc(tslot, 512);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(bars + bFull + i, kLoadWarps * 32 + 1);
            umma::mbar_init(bars + bEmpty + i, 1 + kEpiWarps);
        }
        for (int i = bS; i <= bY; ++i) umma::mbar_init(bars + i, kEpiWarps);
        for (int i = bM1; i <= bEnd; ++i) umma::mbar_init(bars + i, 1);
        umma::fence_mbar_init();
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tm = uniform(*tslot);
    bool ok = true;
    int issued = 0;   // chunks on their way, of the loading threads

    if (warp > kEpiWarps) {
        // ------------------------------------------------------ loading ----
        const int lt = tid - (kEpiWarps + 1) * 32;
        for (int st = 0, turn = 0; issued < chunks; ++issued) {
            const int c = chunks - 1 - issued;
            const long long slot = sq.slot0 + c;
            const unsigned char *up = ws + (size_t)(slot * a.hv + hv) * kUnitBytes;
            const unsigned char *ip = images + (size_t)(slot * a.hk + hk) * L::kTp;
            const T *op = dout + (sq.tok0 + (long long)c * kC) * orow + (long long)hv * a.dv;
            if (c > 0)
                prefetch_stage<T, DKT>(ip - (size_t)a.hk * L::kTp, up - (size_t)a.hv * kUnitBytes, op - kC * orow, orow,
                                       kC, a.dv, lt);
            try_wait(ok, bars + bEmpty + st, (turn & 1) ^ 1);   // the first use needs no wait
            if (!ok) break;
            load_stage<T, DKT>(smem + st * stage_bytes, ip, up, op, orow, sq.len - c * kC, a.dv, lt, bars + bFull + st);
            if (++st == ST) {
                st = 0;
                ++turn;
            }
        }
    } else if (warp == kEpiWarps) {
        // ----------------------------------------------------- products ----
        const uint32_t base = saddr(smem);
        for (int n = 0, st = 0, turn = 0; n < chunks && all_ok(ok); ++n) {
            const int pn = n & 1;
            const uint32_t k0 = base + st * stage_bytes, t0 = k0 + L::kTp;
            // columns 16 ks of dR^T (+)= part p of operand (at, low), K step ib, times part j of T (pt = 0) or PT (1)
            auto t_times = [&](uint32_t at, uint32_t low, int p, int ib, int j, int pt, int ks, bool acc) {
                mma_ts(tm + kTmR + 16 * ks, tm + (p < 2 ? at + 16 * ib + 8 * p : low + 8 * ib),
                       desc_mn(t0 + j * kTpImage + tp_offset(ks) + pt * tp_rows(ks) + (ib - ks) * 256, 128,
                               tp_group(ks)),
                       idesc(16, false, true), acc);
            };
            try_wait(ok, bars + bFull + st, turn & 1);
            // D1 = dS1^T K^T, steps m and NS + m; the orders of the parts' products as in the forward chain
            auto state_times = [&](int m, int most, int least) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int o = most; o >= least; --o)
#pragma unroll
                        for (int j = 0; j < NB; ++j) {
                            if (o - j < 0) continue;
                            const int ks = h * NS + m, p = o - j;
                            mma_ts(tm + kTmK, tm + (p < 2 ? kTmS + 16 * ks + 8 * p : kTmSl + 8 * ks),
                                   desc_k(k0 + j * L::kImg + ks * 4096, 2048, 128), idesc(kC, false, false),
                                   m + h > 0 || o < 2 || j > 0);
                        }
            };
#pragma unroll
            for (int m = 0; m < NS; ++m) {
                try_wait(ok, bars + bS + m, pn);
                umma::fence_after_sync();
                if (elect()) {
                    state_times(m, 2, 1);
                    if (m == NS - 1) {
#pragma unroll
                        for (int i = 0; i < NS; ++i) state_times(i, 0, 0);
                        umma::commit(bars + bM1);
                    }
                }
                __syncwarp();
            }
            // dR^T = dO^T PT + ..
            try_wait(ok, bars + bX, pn);
            umma::fence_after_sync();
            if (elect()) {
#pragma unroll
                for (int o = 2; o >= 0; --o)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                        for (int ib = 3; ib >= ks; --ib)
#pragma unroll
                            for (int p = 0; p < NB; ++p)
                                if (o - p >= 0) t_times(kTmX, kTmXl, p, ib, o - p, 1, ks, ib < 3 || o < 2 || p > 0);
                umma::commit(bars + bMx);
            }
            __syncwarp();
            // .. + (beta e^(G_C - G) D1) T
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                try_wait(ok, bars + bK + m, pn);
                umma::fence_after_sync();
                if (elect()) {
                    auto group = [&](int first, int most, int least) {
#pragma unroll
                        for (int o = most; o >= least; --o)
#pragma unroll
                            for (int ib = first; ib < 4; ib += 2)
#pragma unroll
                                for (int ks = 0; ks <= ib; ++ks)
#pragma unroll
                                    for (int p = 0; p <= o; ++p) t_times(kTmK, kTmKl, p, ib, o - p, 0, ks, true);
                    };
                    group(m, 2, 1);
                    if (m == 1) {
                        group(0, 0, 0);
                        group(1, 0, 0);
                    }
                    if (m == 1) umma::commit(bars + bM2);
                }
                __syncwarp();
            }
            // D3 = (scale e^G dO)^T Q - (e^G dR)^T K, in the place of the state gradient's parts
            auto tok_times = [&](uint32_t at, uint32_t low, int row0, int ks, bool first, int most, int least) {
#pragma unroll
                for (int o = most; o >= least; --o)
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        if (o - j < 0) continue;
                        const int p = o - j;
                        mma_ts(tm + kTmS, tm + (p < 2 ? at + 16 * ks + 8 * p : low + 8 * ks),
                               desc_mn(k0 + j * L::kImg + row0 * 16 + ks * 256, 128, 2048), idesc(DKT, false, true),
                               !first || o < 2 || j > 0);
                    }
            };
            try_wait(ok, bars + bY, pn);
            try_wait(ok, bars + bM1, pn);
            umma::fence_after_sync();
            if (elect())
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) tok_times(kTmX, kTmXl, kC, ks, ks == 0, 2, 1);
            __syncwarp();
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                try_wait(ok, bars + bR + m, pn);
                umma::fence_after_sync();
                if (elect()) {
                    tok_times(kTmR, kTmRl, 0, m, false, 2, 1);
                    tok_times(kTmR, kTmRl, 0, 2 + m, false, 2, 1);
                    if (m == 1) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            tok_times(kTmX, kTmXl, kC, ks, false, 0, 0);
                            tok_times(kTmR, kTmRl, 0, ks, false, 0, 0);
                        }
                        umma::commit(bars + bM3);
                        if (n + ST < chunks) umma::commit(bars + bEmpty + st);
                    }
                }
                __syncwarp();
            }
            if (++st == ST) {
                st = 0;
                ++turn;
            }
        }
    } else {
        // ------------------------------------------------- element-wise ----
        const int h = warp >> 2, v = (warp & 3) * 32 + lane;   // half of the columns, value channel
        const uint32_t mine = tm + ((uint32_t)((warp & 3) * 32) << 16);
        const bool vin = v < a.dv;
        float S[HC];
        const size_t st0 = ((size_t)sg.s * a.hv + hv) * a.dk * a.dv + v;
        const float *from = SUM ? nullptr : a.seg ? su.behind(sums, blockIdx.x) + v : dlast ? dlast + st0 : nullptr;
#pragma unroll
        for (int i = 0; i < HC; ++i) {
            const int d = h * HC + i;
            S[i] = from && vin && d < a.dk ? __ldg(from + (size_t)d * a.dv) : 0.0f;
        }
        auto done = [&](int bar) {   // this warp's tensor-memory writes (and reads) before the barrier
            tm_wait_st();
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + bar);
        };
        for (int n = 0, st = 0, turn = 0; n < chunks; ++n) {
            const int pn = n & 1, c = chunks - 1 - n, rows = sq.len - c * kC;
            const unsigned char *sp = smem + st * stage_bytes;
            const float *eg = reinterpret_cast<const float *>(sp + L::kTp + kTpBytes);
            // lanes past dv compute what channel 0 would be; nothing of it is stored
            const T *os = reinterpret_cast<const T *>(sp + L::kV) + (vin ? v : 0);
            const long long unit = (sq.slot0 + c) * a.hv + hv;
#pragma unroll
            for (int m = 0; m < NS; ++m) {
                float x[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = S[16 * m + j];
                tm_split16(mine + kTmS + 16 * (h * NS + m), mine + kTmSl + 8 * (h * NS + m), x);
                done(bS + m);
            }
            if (!SUM && vin) store_state<HC>(keep_ds + (size_t)unit * a.dk * a.dv, S, h, v, a.dk, a.dv);
            try_wait(ok, bars + bFull + st, turn & 1);
#pragma unroll
            for (int m = 0; m < 2; ++m) {   // dO^T
                const int j0 = h * (kC / 2) + 16 * m;
                float x[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = to_f(os[(j0 + j) * a.dv]);
                tm_parts16<NB>(mine + kTmX + j0, mine + kTmXl + j0 / 2, x);
            }
            done(bX);
            try_wait(ok, bars + bM1, pn);
            umma::fence_after_sync();
#pragma unroll
            for (int m = 0; m < 2; ++m) {   // beta e^(G_C - G) D1
                const int j0 = h * (kC / 2) + 16 * m;
                float x[16], e[16];
                get16(eg + kC + j0, e);
                tm_ld16(mine + kTmK + j0, x);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] *= e[j];
                tm_split16(mine + kTmK + j0, mine + kTmKl + j0 / 2, x);
                done(bK + m);
            }
            if (!all_ok(ok)) break;
            try_wait(ok, bars + bMx, pn);
            umma::fence_after_sync();
#pragma unroll
            for (int m = 0; m < 2; ++m) {   // scale e^G dO^T, in the place of dO^T
                const int j0 = h * (kC / 2) + 16 * m;
                float x[16], e[16];
                get16(eg + j0, e);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = to_f(os[(j0 + j) * a.dv]) * (a.scale * e[j]);
                tm_split16(mine + kTmX + j0, mine + kTmXl + j0 / 2, x);
            }
            done(bY);
            try_wait(ok, bars + bM2, pn);
            umma::fence_after_sync();
#pragma unroll
            for (int m = 0; m < 2; ++m) {   // dR^T = dV^T, and -e^G dR as the next operand
                const int j0 = h * (kC / 2) + 16 * m;
                float x[16], e[16];
                get16(eg + j0, e);
                tm_ld16(mine + kTmR + j0, x);
                float y[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) y[j] = -e[j] * x[j];
                tm_split16(mine + kTmR + j0, mine + kTmRl + j0 / 2, y);
                done(bR + m);
                if (SUM) continue;
                if (vin) store_tokens(keep_dr + (size_t)unit * kC * a.dv, x, j0, v);
                store16<T>(dv + (sq.tok0 + (long long)c * kC + j0) * orow + (long long)hv * a.dv + v, orow, x, lane, vin,
                           rows - j0);
            }
            const float total = eg[kC - 1];   // e^(G_C): rows past the end have g = 0
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + bEmpty + st);
            try_wait(ok, bars + bM3, pn);
            umma::fence_after_sync();
#pragma unroll
            for (int i = 0; i < HC; i += 16) {
                float x[16];
                tm_ld16(mine + kTmS + h * HC + i, x);
#pragma unroll
                for (int j = 0; j < 16; ++j) S[i + j] = fmaf(total, S[i + j], x[j]);
            }
            if (++st == ST) {
                st = 0;
                ++turn;
            }
        }
        float *to = SUM ? su.dn(sums, blockIdx.x) + v : dinit && sg.index == 0 ? dinit + st0 : nullptr;
        if (to && vin) {
#pragma unroll
            for (int i = 0; i < HC; ++i)
                if (h * HC + i < a.dk) to[(size_t)(h * HC + i) * a.dv] = S[i];
        }
    }
    if (!ok && flags) atomicOr(flags, S4_FLAG_TIMEOUT);
    umma::fence_before_sync();
    if (__syncthreads_or(!ok)) {   // a wait ran out: what is still under way ends before its memory goes
        if (warp > kEpiWarps) drain_copies(bars + bFull, issued, ST);
        if (warp == kEpiWarps) {
            if (elect()) umma::commit(bars + bEnd);
            __syncwarp();
            umma::mbar_wait(bars + bEnd, 0, kDrainLimit);
        }
        __syncthreads();
    }
    umma::fence_after_sync();
    if (warp == 0) umma::tmem_dealloc(tm, 512);
}

template <typename T, int DKT>
cudaError_t run(const DeltaArgs &a, const void *dout, const float *dlast, float *dinit, const void *ws, void *dv,
                float *keep_ds, float *keep_dr, void *summaries, unsigned *flags, cudaStream_t st) {
    const int smem = Stage<T, DKT>::count(a.dv) * Stage<T, DKT>::bytes(a.dv) + 256;
    static SmemLimit limit, limit_sum;
    cudaError_t e = limit.raise(k_delta_backward<T, DKT, false>, smem);
    if (e != cudaSuccess) return e;
    const long long chunks = slots(a.tokens, a.n), blocks = segments(chunks, a.n, a.seg) * a.hv;
    const unsigned char *units = (const unsigned char *)ws, *images = units + (size_t)chunks * a.hv * kUnitBytes;
    float *sums = (float *)summaries;
    if (a.seg) {
        e = limit_sum.raise(k_delta_backward<T, DKT, true>, smem);
        if (e != cudaSuccess) return e;
        k_delta_backward<T, DKT, true><<<(unsigned)blocks, kThreads, smem, st>>>(
            a, (const T *)dout, nullptr, nullptr, sums, units, images, nullptr, nullptr, nullptr, flags);
        e = launch_delta_join(a, dlast, sums, true, true, flags, st);
        if (e != cudaSuccess) return e;
    }
    k_delta_backward<T, DKT, false><<<(unsigned)blocks, kThreads, smem, st>>>(
        a, (const T *)dout, dlast, dinit, sums, units, images, (T *)dv, keep_ds, keep_dr, flags);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_backward(int dtype, const DeltaArgs &a, const void *dout, const float *dlast, float *dinit,
                                  const void *ws, void *dv, float *keep_ds, float *keep_dr, void *summaries,
                                  unsigned *flags, cudaStream_t st) {
    const bool wide = a.dk > 64;
    if (dtype == S4_BF16)
        return wide ? run<__nv_bfloat16, 128>(a, dout, dlast, dinit, ws, dv, keep_ds, keep_dr, summaries, flags, st)
                    : run<__nv_bfloat16, 64>(a, dout, dlast, dinit, ws, dv, keep_ds, keep_dr, summaries, flags, st);
    if (dtype == S4_F16)
        return wide ? run<__half, 128>(a, dout, dlast, dinit, ws, dv, keep_ds, keep_dr, summaries, flags, st)
                    : run<__half, 64>(a, dout, dlast, dinit, ws, dv, keep_ds, keep_dr, summaries, flags, st);
    return wide ? run<float, 128>(a, dout, dlast, dinit, ws, dv, keep_ds, keep_dr, summaries, flags, st)
                : run<float, 64>(a, dout, dlast, dinit, ws, dv, keep_ds, keep_dr, summaries, flags, st);
}

}  // namespace s4
