// delta_chunk.cu -- the chunked gated delta rule, forward: one block walks the
// chunks of one sequence and value head with the state in registers.
//
// Everything is kept transposed, value channel = tensor-memory lane, so that
// the three products of a chunk that depend on each other take their left
// operand from tensor memory, written there by the threads that computed it,
// and their right operand from the natural image of [K; Q] or [T; PT]:
//     D1 = S0^T [K; Q]^T                           (128 x 128)
//     R^T = V^T - e^G D1k,   D2 = R^T [T; PT]^T    (E^T and (PT R)^T)
//     D3 = (beta e^(G_C - G) E)^T K                (128 x Dk)
//     S1^T = e^(G_C) S0^T + D3,   O^T = scale e^G D1q + (PT R)^T.
// Roles: warps 0-7 the element-wise steps (two warps per lane quarter, each
// half the columns), warp 8 issues the products, warps 9-11 load.
//
// What bounds it: the chain of a chunk, three products and three element-wise
// passes one after the other, most of it the splitting in the passes. A
// product starts with the first 16 columns of its operand; Q's and PT's
// products and the output run in the chain's gaps. A block needs all 512
// tensor-memory columns, so there is one per SM. Measured: 4 x 4096 tokens, 32
// heads of 128 bf16 (128 chains of 64 chunks) 235 us, 3.7 us a chunk; 327 us
// when the states and E are kept for the backward pass (0.8 GB more to write).
#include "delta.cuh"
#include "s4dplr.h"

#include <cmath>

namespace s4 {
namespace {

using namespace delta;

// Tensor-memory columns. An operand's high and middle parts take the place of
// the accumulator it was computed from, 16 columns by 16 columns, so a warp
// overwrites only what it alone has read:
//   kTmS   the state's parts, D3 in their place (128), low parts at kTmSl
//   kTmK   S0^T K^T (64), then R's parts, low ones at kTmRl
//   kTmE   E^T (64), then the parts of beta e^(G_C - G) E, low ones at kTmEl
//   kTmQ, kTmO   S0^T Q^T and (PT R)^T (64 each)
constexpr int kTmS = 0, kTmSl = 128, kTmK = 192, kTmE = 256, kTmQ = 320, kTmO = 384, kTmRl = 448, kTmEl = 480;

enum { bFull = 0, bEmpty = 2, bS = 4, bR = 8, bE = 10, bO = 12, bM1, bM2, bMq, bM2o, bM3, bEnd, bCount };

// SUM: what a segment does to the state, S -> M S + N, without output: blocks
// 2 b write N (the segment from a zero state), blocks 2 b + 1 M (without V,
// from the identity; lanes are M's columns). Otherwise the segment itself, from
// the state that `starts` has for it.
template <typename T, int DKT, bool SUM>
__global__ void __launch_bounds__(kThreads, 1) k_delta_forward(DeltaArgs a, const float *init, float *last,
                                                               float *sums, bool keep_m,
                                                               const unsigned char *ws,
                                                               const unsigned char *images, float *keep_s,
                                                               float *keep_e, unsigned *flags) {
    using L = Stage<T, DKT>;
    constexpr int NB = Parts<T>::n, HC = DKT / 2, NS = DKT / 32;   // NS: K steps of a half of the state
    extern __shared__ __align__(1024) unsigned char smem[];
    const int ST = L::count(a.dv), stage_bytes = L::bytes(a.dv);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + ST * stage_bytes);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + bCount);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const unsigned block = SUM ? blockIdx.x >> 1 : blockIdx.x;
    const bool ident = SUM && (blockIdx.x & 1);
    const int hv = block % a.hv, hk = hv / (a.hv / a.hk);
    const Segment sg = segment_of(a, block / a.hv);
    // not needed: the last segment's N, its M unless for the way back, and the
    // first one's M where it would meet zeros
    if (sg.s < 0 || (SUM && sg.last && !(ident && keep_m && sg.index > 0))) return;
    if (ident && sg.index == 0 && !init) return;
    const Summaries su(a.dk, a.dv, keep_m);
    Seq sq = sequence(a, sg.s);   // from here on the segment as a sequence
    sq.tok0 += (long long)sg.first * kC;
    sq.slot0 += sg.first;
    sq.len = sq.len - sg.first * kC < sg.chunks * kC ? sq.len - sg.first * kC : sg.chunks * kC;
    const int chunks = uniform(sg.chunks);
    const int dv = ident ? a.dk : a.dv;   // lanes in use

    if (warp == 0) umma::tmem_alloc(tslot, 512);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(bars + bFull + i, kLoadWarps * 32 + 1);
            umma::mbar_init(bars + bEmpty + i, 1 + kEpiWarps);
        }
        for (int i = bS; i <= bO; ++i) umma::mbar_init(bars + i, kEpiWarps);
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
            const int c = issued;
            const long long slot = sq.slot0 + c;
            const unsigned char *up = ws + (size_t)(slot * a.hv + hv) * kUnitBytes;
            const unsigned char *ip = images + (size_t)(slot * a.hk + hk) * L::kTp;
            const T *vp = (const T *)a.v + (sq.tok0 + (long long)c * kC) * a.sv + (long long)hv * a.dv;
            if (c + 1 < chunks)
                prefetch_stage<T, DKT>(ip + (size_t)a.hk * L::kTp, up + (size_t)a.hv * kUnitBytes, vp + kC * a.sv, a.sv,
                                       sq.len - (c + 1) * kC, a.dv, lt);
            try_wait(ok, bars + bEmpty + st, (turn & 1) ^ 1);   // the first use needs no wait
            if (!ok) break;
            load_stage<T, DKT>(smem + st * stage_bytes, ip, up, vp, a.sv, sq.len - c * kC, a.dv, lt, bars + bFull + st);
            if (++st == ST) {
                st = 0;
                ++turn;
            }
        }
    } else if (warp == kEpiWarps) {
        // ----------------------------------------------------- products ----
        // A K step's products start as soon as the threads have written its
        // parts. What the next step waits for goes first, Q's and PT's products
        // into the gaps.
        const uint32_t base = saddr(smem);
        for (int c = 0, st = 0, turn = 0; c < chunks && all_ok(ok); ++c) {
            const int pc = c & 1;
            const uint32_t k0 = base + st * stage_bytes, t0 = k0 + L::kTp;
            // Of every product the orders from `most` to `least` (2: the smallest
            // parts' products). The accumulators round down with every
            // addition, so the largest products come last of all steps.
            // S0^T K^T (row0 = 0) or S0^T Q^T (64): steps n and NS + n
            auto state_times = [&](uint32_t d, int row0, int n, int most, int least) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int o = most; o >= least; --o)
#pragma unroll
                        for (int j = 0; j < NB; ++j) {
                            if (o - j < 0) continue;
                            const int ks = h * NS + n, p = o - j;
                            mma_ts(tm + d, tm + (p < 2 ? kTmS + 16 * ks + 8 * p : kTmSl + 8 * ks),
                                   desc_k(k0 + j * L::kImg + ks * 4096 + row0 * 16, 2048, 128),
                                   idesc(kC, false, false), n + h > 0 || o < 2 || j > 0);
                        }
            };
            // R^T T^T (pt = 0) or R^T PT^T (1): steps n and 2 + n, which meet rows 16 ks and up
            auto r_times = [&](uint32_t d, int pt, int n, int most, int least) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int o = most; o >= least; --o)
#pragma unroll
                        for (int j = 0; j <= o; ++j) {
                            const int ks = 2 * h + n, p = o - j;
                            mma_ts(tm + d + 16 * ks, tm + (p < 2 ? kTmK + 16 * ks + 8 * p : kTmRl + 8 * ks),
                                   desc_k(t0 + j * kTpImage + tp_offset(ks) + pt * tp_rows(ks), tp_group(ks), 128),
                                   idesc(kC - 16 * ks, false, false), n + h > 0 || o < 2 || j > 0);
                        }
            };
            // D3 = (beta e^(G_C - G) E)^T K, in the place of the state's parts
            auto e_times = [&](int n, int most, int least) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int o = most; o >= least; --o)
#pragma unroll
                        for (int j = 0; j < NB; ++j) {
                            if (o - j < 0) continue;
                            const int ks = 2 * h + n, p = o - j;
                            mma_ts(tm + kTmS, tm + (p < 2 ? kTmE + 16 * ks + 8 * p : kTmEl + 8 * ks),
                                   desc_mn(k0 + j * L::kImg + ks * 256, 128, 2048), idesc(DKT, false, true),
                                   n + h > 0 || o < 2 || j > 0);
                        }
            };
            try_wait(ok, bars + bFull + st, turn & 1);
            if (c > 0) try_wait(ok, bars + bM2o, pc ^ 1);   // R's parts have been read
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                try_wait(ok, bars + bS + n, pc);
                umma::fence_after_sync();
                if (elect()) {
                    state_times(kTmK, 0, n, 2, 1);
                    if (n == NS - 1) {
#pragma unroll
                        for (int i = 0; i < NS; ++i) state_times(kTmK, 0, i, 0, 0);
                        umma::commit(bars + bM1);
                    }
                }
                __syncwarp();
            }
            if constexpr (!SUM) {
                if (c > 0) try_wait(ok, bars + bO, pc ^ 1);   // the last output's terms have been read
                umma::fence_after_sync();
                if (elect())
#pragma unroll
                    for (int n = 0; n < NS; ++n) state_times(kTmQ, kC, n, 2, 1);
                __syncwarp();
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                try_wait(ok, bars + bR + n, pc);
                umma::fence_after_sync();
                if (elect()) {
                    r_times(kTmE, 0, n, 2, 1);
                    if (n == 1) {
                        r_times(kTmE, 0, 0, 0, 0);
                        r_times(kTmE, 0, 1, 0, 0);
                        umma::commit(bars + bM2);
                        if constexpr (!SUM) {
#pragma unroll
                            for (int i = 0; i < NS; ++i) state_times(kTmQ, kC, i, 0, 0);
                        }
                        umma::commit(bars + bMq);
                    }
                }
                __syncwarp();
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                try_wait(ok, bars + bE + n, pc);
                if (n == 0) try_wait(ok, bars + bMq, pc);   // the state's parts have been read
                umma::fence_after_sync();
                if (elect()) {
                    e_times(n, 2, 1);
                    if (n == 1) {
                        e_times(0, 0, 0);
                        e_times(1, 0, 0);
                        umma::commit(bars + bM3);
                        if constexpr (!SUM) {
                            r_times(kTmO, 1, 0, 2, 1);
                            r_times(kTmO, 1, 1, 2, 1);
                            r_times(kTmO, 1, 0, 0, 0);
                            r_times(kTmO, 1, 1, 0, 0);
                        }
                        umma::commit(bars + bM2o);
                        if (c + ST < chunks) umma::commit(bars + bEmpty + st);
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
        const bool vin = v < dv;
        const long long orow = (long long)a.hv * a.dv;
        float S[HC];
        const size_t st0 = ((size_t)sg.s * a.hv + hv) * a.dk * a.dv + v;
        const float *from = a.seg ? su.start(sums, block) + v : init ? init + st0 : nullptr;
#pragma unroll
        for (int i = 0; i < HC; ++i) {
            const int d = h * HC + i;
            if (SUM)
                S[i] = ident && d == v && vin ? 1.0f : 0.0f;
            else
                S[i] = from && vin && d < a.dk ? __ldg(from + (size_t)d * a.dv) : 0.0f;
        }
        auto done = [&](int bar) {   // this warp's tensor-memory writes (and reads) before the barrier
            tm_wait_st();
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + bar);
        };
        auto put_state = [&]() {
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                float x[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = S[16 * n + j];
                tm_split16(mine + kTmS + 16 * (h * NS + n), mine + kTmSl + 8 * (h * NS + n), x);
                done(bS + n);
            }
        };
        // O^T = scale e^G S0^T Q^T + (PT R)^T of chunk c, in stage st
        auto put_output = [&](int c, int st) {
            const int rows = sq.len - c * kC < kC ? sq.len - c * kC : kC;
            const float *eg = reinterpret_cast<const float *>(smem + st * stage_bytes + L::kTp + kTpBytes);
            try_wait(ok, bars + bM2o, c & 1);
            umma::fence_after_sync();
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int j0 = h * (kC / 2) + 16 * n;
                float x[16], y[16], e[16];
                get16(eg + j0, e);
                tm_ld16(mine + kTmQ + j0, x);
                tm_ld16(mine + kTmO + j0, y);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = fmaf(a.scale * e[j], x[j], y[j]);
                store16<T>((T *)a.o + (sq.tok0 + (long long)c * kC + j0) * orow + (long long)hv * a.dv + v, orow, x,
                           lane, vin, rows - j0);
            }
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bars + bO);
                mbar_arrive(bars + bEmpty + st);
            }
        };
        if (chunks) put_state();
        [[maybe_unused]] int before = 0;
        for (int c = 0, st = 0, turn = 0; c < chunks; ++c) {
            const int pc = c & 1;
            const unsigned char *sp = smem + st * stage_bytes;
            const float *eg = reinterpret_cast<const float *>(sp + L::kTp + kTpBytes);
            // lanes past dv compute what channel 0 would be; nothing of it is stored
            const T *vs = reinterpret_cast<const T *>(sp + L::kV) + (v < a.dv ? v : 0);
            const long long unit = (sq.slot0 + c) * a.hv + hv;
            if (!SUM && keep_s && vin) store_state<HC>(keep_s + (size_t)unit * a.dk * a.dv, S, h, v, a.dk, a.dv);
            if (!SUM && c > 0) put_output(c - 1, before);
            try_wait(ok, bars + bFull + st, turn & 1);
            try_wait(ok, bars + bM1, pc);
            umma::fence_after_sync();
#pragma unroll
            for (int n = 0; n < 2; ++n) {   // R^T = V^T - e^G S0^T K^T
                const int j0 = h * (kC / 2) + 16 * n;
                float x[16], e[16], r[16];
                get16(eg + j0, e);
#pragma unroll
                for (int j = 0; j < 16; ++j) r[j] = ident ? 0.0f : to_f(vs[(j0 + j) * a.dv]);
                tm_ld16(mine + kTmK + j0, x);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = fmaf(-e[j], x[j], r[j]);
                tm_split16(mine + kTmK + j0, mine + kTmRl + j0 / 2, x);
                done(bR + n);
            }
            try_wait(ok, bars + bM2, pc);
            umma::fence_after_sync();
#pragma unroll
            for (int n = 0; n < 2; ++n) {   // E^T, and beta e^(G_C - G) E as the next operand
                const int j0 = h * (kC / 2) + 16 * n;
                float x[16], e[16];
                get16(eg + kC + j0, e);
                tm_ld16(mine + kTmE + j0, x);
                if (!SUM && keep_e && vin) store_tokens(keep_e + (size_t)unit * kC * a.dv, x, j0, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] *= e[j];
                tm_split16(mine + kTmE + j0, mine + kTmEl + j0 / 2, x);
                done(bE + n);
            }
            const float total = eg[kC - 1];   // e^(G_C): rows past the end have g = 0
            if (!all_ok(ok)) break;
            if (SUM && lane == 0) mbar_arrive(bars + bEmpty + st);
            try_wait(ok, bars + bM3, pc);
            umma::fence_after_sync();
#pragma unroll
            for (int i = 0; i < HC; i += 16) {
                float x[16];
                tm_ld16(mine + kTmS + h * HC + i, x);
#pragma unroll
                for (int j = 0; j < 16; ++j) S[i + j] = fmaf(total, S[i + j], x[j]);
            }
            if (c + 1 < chunks) put_state();
            before = st;
            if (++st == ST) {
                st = 0;
                ++turn;
            }
        }
        if constexpr (SUM) {
            if (chunks) try_wait(ok, bars + bM2o, (chunks - 1) & 1);   // its arrival, which only a next chunk waits for
            float *to = ident ? su.m(sums, block) + (size_t)v * a.dk : su.n(sums, block) + v;
            float *rows = ident && keep_m ? su.m_rows(sums, block) + v : nullptr;
            if (vin)
#pragma unroll
                for (int i = 0; i < HC; ++i)
                    if (h * HC + i < a.dk) {
                        to[(size_t)(h * HC + i) * (ident ? 1 : a.dv)] = S[i];
                        if (rows) rows[(size_t)(h * HC + i) * a.dk] = S[i];
                    }
        } else {
            if (chunks && all_ok(ok)) put_output(chunks - 1, before);
            if (last && sg.last && vin) {
#pragma unroll
                for (int i = 0; i < HC; ++i)
                    if (h * HC + i < a.dk) last[st0 + (size_t)(h * HC + i) * a.dv] = S[i];
            }
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
cudaError_t run(const DeltaArgs &a, const float *init, float *last, const void *ws, float *keep_s, float *keep_e,
                void *summaries, unsigned *flags, cudaStream_t st) {
    const int smem = Stage<T, DKT>::count(a.dv) * Stage<T, DKT>::bytes(a.dv) + 256;
    static SmemLimit limit, limit_sum;
    cudaError_t e = limit.raise(k_delta_forward<T, DKT, false>, smem);
    if (e != cudaSuccess) return e;
    const long long chunks = slots(a.tokens, a.n), blocks = segments(chunks, a.n, a.seg) * a.hv;
    const unsigned char *units = (const unsigned char *)ws, *images = units + (size_t)chunks * a.hv * kUnitBytes;
    float *sums = (float *)summaries;
    const bool keep = keep_s != nullptr;
    if (a.seg) {
        e = limit_sum.raise(k_delta_forward<T, DKT, true>, smem);
        if (e != cudaSuccess) return e;
        k_delta_forward<T, DKT, true><<<(unsigned)(2 * blocks), kThreads, smem, st>>>(a, init, nullptr, sums, keep, units,
                                                                                    images, nullptr, nullptr, flags);
        e = launch_delta_join(a, init, sums, keep, false, flags, st);
        if (e != cudaSuccess) return e;
    }
    k_delta_forward<T, DKT, false><<<(unsigned)blocks, kThreads, smem, st>>>(a, init, last, sums, keep, units, images,
                                                                            keep_s, keep_e, flags);
    return cudaGetLastError();
}

}  // namespace

// Few long chains leave most SMs idle: then every sequence is cut into segments,
// what each does to the state is computed for all at once (twice the chain's
// work: M and N), joined, and the segments run again from their states. Times
// in chunks of a chain (3.1 us; M and N without output 0.85 of that, a join
// 0.8, the extra launches 4). Lengths of packed sequences are not known here;
// the longest is taken as it is on average when `tokens` are cut at random
// places, H_n / n of them (H_n the harmonic number): 8192 tokens in sequences
// of 4000, 500, 1000, 692 and four of 500, 8 heads, 314 us in one piece each
// and 138 in segments; where all have 1024, 88 and 126. One sequence of
// 65536 tokens, 8 heads of 128: 3515 us for the whole call in one piece, 890
// us in 18.
//
// A workspace for many tokens has to serve calls with fewer. The best number of
// segments goes up and down with the length where they are a few chunks each
// and the last is not full. Without that rounding a number's time is a line in
// the length, steeper and from a lower start the fewer they are, so the best
// one only rises with the length. Up to a quarter more than that may be taken
// (the rule finds its best among them in 99 of 100 lengths, and within 4% in
// the others), and room is kept for as many: at most n most / cuts + 2 n.
int delta_segment(long long tokens, int n, int hv, bool packed, long long *count) {
    constexpr double kSms = 148;
    constexpr int kMost = 64;
    const double all = (double)tokens / kC, cuts = packed && n > 1 ? log((double)n) + 0.577 + 0.5 / n : 1;
    // the longest sequence, and how many as long make up all tokens
    const double c = ceil(all / n * cuts), chains = n / cuts * hv, one = 0.9 * ceil(chains / kSms) * c;
    double per[kMost + 1], best = one;   // per: time by chunks of a segment
    int unrounded = 0;
    for (int k = 3; k <= kMost && k <= c; ++k) {
        per[k] = 0.85 * ceil(2 * chains * (k - 1) / kSms) + ceil(chains * k / kSms);
        const double t = per[k] * c / k + 0.8 * k + 4;
        if (t < best) {
            best = t;
            unrounded = k;
        }
    }
    const int most = (5 * unrounded + 3) / 4;
    int seg = 0;
    best = one;
    for (int k = 3; k <= most && k <= kMost && k <= c; ++k) {
        const double len = ceil(c / k), t = per[k] * len + 0.8 * k + 4;
        if (t < best) {
            best = t;
            seg = (int)len;
        }
    }
    *count = most ? (long long)ceil(n * most / cuts) + 2 * (long long)n : 0;
    const long long used = seg ? segments(slots(tokens, n), n, seg) : 0;
    if (*count < used) *count = used;
    return seg;
}

size_t delta_segment_bytes(long long count, int hv, int dk, int dv, bool keep) {
    return (size_t)count * hv * Summaries(dk, dv, keep).unit() * sizeof(float);
}

cudaError_t launch_delta_forward(int dtype, const DeltaArgs &a, const float *init, float *last, const void *ws,
                                 float *keep_s, float *keep_e, void *summaries, unsigned *flags, cudaStream_t st) {
    const bool wide = a.dk > 64;
    if (dtype == S4_BF16)
        return wide ? run<__nv_bfloat16, 128>(a, init, last, ws, keep_s, keep_e, summaries, flags, st)
                    : run<__nv_bfloat16, 64>(a, init, last, ws, keep_s, keep_e, summaries, flags, st);
    if (dtype == S4_F16)
        return wide ? run<__half, 128>(a, init, last, ws, keep_s, keep_e, summaries, flags, st)
                    : run<__half, 64>(a, init, last, ws, keep_s, keep_e, summaries, flags, st);
    return wide ? run<float, 128>(a, init, last, ws, keep_s, keep_e, summaries, flags, st)
                : run<float, 64>(a, init, last, ws, keep_s, keep_e, summaries, flags, st);
}

}  // namespace s4
