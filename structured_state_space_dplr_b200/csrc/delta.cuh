// delta.cuh -- what the kernels of the chunked gated delta rule share: the
// geometry of chunks, the operand images, the split of a float into three
// bf16 parts and the tensor-core wrappers that umma.cuh does not have.
//
// A chunk is 64 tokens of one sequence. With G the running sum of g in the
// chunk, S0 the state before it and D_b = diag(beta):
//     A_ij = e^(G_i - G_j) k_i.k_j (j < i),      T = (I + A D_b)^-1,
//     P_ij = scale e^(G_i - G_j) q_i.k_j (j <= i), PT = P D_b T,
//     R = V - e^G K S0,   E = T R,   (u = beta E)
//     O = scale e^G Q S0 + PT R,
//     S1 = e^(G_C) S0 + (e^(G_C - G) K)^T D_b E.
// The rows past a sequence's end take part with k = q = v = 0, beta = 0 and
// g = 0 and change nothing.
//
// Precision: every product runs on the bf16 tensor cores with float
// accumulators. An operand that is not bf16 already is split into three bf16
// parts (24 bits, the parts' exponents as wide as float's), and the products
// of parts whose order is at least 2^-16 are summed; a bf16 input is one part, a
// half two. A product is off by up to 2^-23 for the orders left out and 2^-23
// for the accumulator, which truncates, where a float product has 2^-24: results
// are off by about twice what they are in float arithmetic (float training
// against 64 bits: 6e-7 relative, 3e-7), at any scale of the values up to
// bf16's largest (3.39e38; larger floats become infinities).
//
// Operand image: a matrix of `rows` rows in 8 x 8 blocks of 128 bytes (row by
// row, 16 bytes each), blocks of one column group one after the other. The
// same image serves as K-major operand (rows are M or N, columns K) and as
// MN-major operand (columns are M or N, rows K).
#pragma once

#include "dtype.cuh"
#include "launch.h"
#include "umma.cuh"

namespace s4 {
namespace delta {

constexpr int kC = 64;                         // tokens of a chunk
// One part of T and PT in the workspace. Both are lower triangular: the 16
// columns of step ks have rows 16 ks and up only, two column groups of 64 - 16
// ks rows of T and then as many of PT.
constexpr int kTpImage = 10240;
constexpr int kTpBytes = 3 * kTpImage;
__host__ __device__ constexpr int tp_offset(int ks) { return 4096 * ks - 512 * ks * (ks - 1); }
__host__ __device__ constexpr int tp_rows(int ks) { return (kC - 16 * ks) * 16; }      // bytes: T's rows of a group
__host__ __device__ constexpr int tp_group(int ks) { return 2 * tp_rows(ks); }         // bytes of a column group
constexpr int kFacBytes = 2 * kC * 4;          // e^G and beta e^(G_C - G)
constexpr int kUnitBytes = kTpBytes + kFacBytes;   // workspace of one chunk and value head
constexpr uint32_t kSpinLimit = 1u << 22;      // polls of a wait
constexpr uint32_t kDrainLimit = 1u << 16;     // of a wait for what is in flight at a block's end

// parts that an input of the type is exactly the sum of (float: to 24 bits)
template <typename T> struct Parts { static constexpr int n = 3; };
template <> struct Parts<__nv_bfloat16> { static constexpr int n = 1; };
template <> struct Parts<__half> { static constexpr int n = 2; };

// ------------------------------------------------------------ geometry ----
struct Seq {
    long long tok0, slot0;   // first token, first chunk slot
    int len;
};
// Offsets outside [0, tokens] or out of order are clamped: a bad cu gives bad
// numbers, never an access out of range.
__device__ __forceinline__ Seq sequence(const DeltaArgs &a, int s) {
    Seq r;
    if (a.cu) {
        long long lo = __ldg(a.cu + s), hi = __ldg(a.cu + s + 1);
        lo = lo < 0 ? 0 : lo > a.tokens ? a.tokens : lo;
        hi = hi < lo ? lo : hi > a.tokens ? a.tokens : hi;
        r.tok0 = lo;
        r.len = (int)(hi - lo);
    } else {
        r.tok0 = (long long)s * a.t;
        r.len = a.t;
    }
    // distinct for distinct (sequence, chunk): floor(x) + ceil(y) <= floor(x + y) + 1
    r.slot0 = r.tok0 / kC + s;
    return r;
}
// Segments: a.seg chunks of one sequence (the last one fewer), or the whole
// sequence; every sequence has one at least. Numbered like the slots.
__host__ __device__ inline long long segments(long long slots, int n, int seg) { return (seg ? slots / seg : 0) + n; }
struct Segment {
    int s, index;            // sequence (-1: no such segment), number in it
    int first, chunks;       // first chunk and chunks (none of an empty sequence)
    bool last;               // the sequence's last
};
__device__ __forceinline__ long long segment0(const DeltaArgs &a, int s) {
    return (a.seg ? sequence(a, s).slot0 / a.seg : 0) + s;
}
__device__ __forceinline__ Segment segment_of(const DeltaArgs &a, long long number) {
    Segment r;
    r.s = 0;
    if (a.seg == 0) {
        r.s = (int)number;
    } else {
        for (int lo = 0, hi = a.n; lo < hi;) {
            const int m = (lo + hi) >> 1;
            if (segment0(a, m) <= number) {
                r.s = m;
                lo = m + 1;
            } else {
                hi = m;
            }
        }
    }
    const int all = (sequence(a, r.s).len + kC - 1) / kC, len = a.seg ? a.seg : all;
    const long long index = a.seg ? number - segment0(a, r.s) : 0;
    if (index < 0 || (index > 0 && index * len >= all)) r.s = -1;
    r.index = (int)index;
    r.first = r.index * len;
    r.chunks = all - r.first < len ? all - r.first : len;
    r.last = r.first + r.chunks >= all;
    return r;
}

// What is kept of segments, all in float: for each segment and value head N
// [dk][dv] and M [dk][dk] by columns (a segment takes the state S to M S + N),
// and the state before it; with `keep`, for the backward pass, M by rows, the
// gradient dN [dk][dv] (the state's gradient goes back as M^T dS + dN) and the
// state's gradient behind it.
struct Summaries {
    size_t dd, dv;   // floats of M and of a state
    bool keep;
    __host__ __device__ Summaries(int dk, int dv_, bool keep_) : dd((size_t)dk * dk), dv((size_t)dk * dv_), keep(keep_) {}
    __host__ __device__ size_t unit() const { return 2 * dv + dd + (keep ? dd + 2 * dv : 0); }
    __host__ __device__ float *n(float *p, size_t u) const { return p + u * unit(); }
    __host__ __device__ float *m(float *p, size_t u) const { return n(p, u) + dv; }
    __host__ __device__ float *start(float *p, size_t u) const { return m(p, u) + dd; }
    __host__ __device__ float *m_rows(float *p, size_t u) const { return start(p, u) + dv; }
    __host__ __device__ float *dn(float *p, size_t u) const { return m_rows(p, u) + dd; }
    __host__ __device__ float *behind(float *p, size_t u) const { return dn(p, u) + dv; }
};

// the chunk that owns a slot: its first token and its tokens (0: none)
struct Chunk {
    long long tok;
    int rows;
};
__device__ __forceinline__ Chunk chunk_of(const DeltaArgs &a, long long slot) {
    int s = 0;   // the last sequence that starts at or before the slot
    for (int lo = 0, hi = a.n; lo < hi;) {
        const int m = (lo + hi) >> 1;
        if (sequence(a, m).slot0 <= slot) {
            s = m;
            lo = m + 1;
        } else {
            hi = m;
        }
    }
    const Seq sq = sequence(a, s);
    const long long c0 = (slot - sq.slot0) * kC;
    Chunk c;
    c.tok = sq.tok0 + c0;
    c.rows = c0 < 0 || c0 >= sq.len ? 0 : sq.len - c0 < kC ? (int)(sq.len - c0) : kC;
    return c;
}

// Running sums of g over the chunk, in units of ln 2 and in double (differences
// of large sums keep float's accuracy), by one warp: lane l has the tokens 2 l
// (x, b0 = its beta) and 2 l + 1 (y, b1); tokens past `rows` have g = beta = 0.
struct GateSums {
    double x, y;
    float b0, b1;
};
__device__ __forceinline__ GateSums gate_sums(const DeltaArgs &a, long long tok, int hv, int rows, int lane) {
    const int j = 2 * lane;
    const long long at = tok * a.hv + hv;
    float g0 = j < rows ? __ldg(a.g + at + (long long)j * a.hv) : 0.0f;
    float g1 = j + 1 < rows ? __ldg(a.g + at + (long long)(j + 1) * a.hv) : 0.0f;
    GateSums r;
    r.b0 = j < rows ? __ldg(a.beta + at + (long long)j * a.hv) : 0.0f;
    r.b1 = j + 1 < rows ? __ldg(a.beta + at + (long long)(j + 1) * a.hv) : 0.0f;
    // exp(-1e5) is 0 as exp(-inf) is, and differences stay numbers
    g0 = g0 < -1e5f ? -1e5f : g0;
    g1 = g1 < -1e5f ? -1e5f : g1;
    constexpr double kLog2e = 1.4426950408889634;   // 1 / ln 2
    const double d1 = (double)g1 * kLog2e;
    double y = (double)g0 * kLog2e + d1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    r.x = y - d1;
    r.y = y;
    return r;
}

__host__ __device__ inline long long slots(long long tokens, int n) { return tokens / kC + n; }

// ---------------------------------------------------------------- split ----
__device__ __forceinline__ float lo_f(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_f(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// two floats at once
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_get(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// a and b as N bf16 parts each, a in the low halves; each part is what the
// ones before it leave, rounded to nearest
template <int N>
__device__ __forceinline__ void split(float a, float b, uint32_t (&p)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p[i] = pack2(a, b);
        if (i + 1 < N) f2_get(f2_sub(f2(a, b), f2(lo_f(p[i]), hi_f(p[i]))), a, b);
    }
}

// 8 elements at p (16-byte aligned) as the parts of their type
__device__ __forceinline__ void load_parts(const __nv_bfloat16 *p, uint4 (&o)[1]) {
    o[0] = __ldg(reinterpret_cast<const uint4 *>(p));
}
__device__ __forceinline__ void load_parts(const __half *p, uint4 (&o)[2]) {
    const uint4 r = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t s[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        split<2>(f.x, f.y, s[i]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) o[j] = make_uint4(s[0][j], s[1][j], s[2][j], s[3][j]);
}
__device__ __forceinline__ void load_parts(const float *p, uint4 (&o)[3]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    uint32_t s[4][3];
    split<3>(a.x, a.y, s[0]);
    split<3>(a.z, a.w, s[1]);
    split<3>(b.x, b.y, s[2]);
    split<3>(b.z, b.w, s[3]);
#pragma unroll
    for (int j = 0; j < 3; ++j) o[j] = make_uint4(s[0][j], s[1][j], s[2][j], s[3][j]);
}

// ------------------------------------------------------- tensor cores ----
using umma::saddr;

// descriptor of an image: `mn` bytes between 8-row groups of M or N, `k` between those of K
__device__ __forceinline__ uint64_t desc_k(uint32_t addr, uint32_t k, uint32_t mn) {   // K-major
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(k >> 4) << 16) | ((uint64_t)(mn >> 4) << 32) |
           ((uint64_t)1 << 46);
}
// MN-major without swizzle has the same two fields
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t k, uint32_t mn) { return desc_k(addr, k, mn); }

// bf16 x bf16 -> f32, M = 128, N; A K-major (or from tensor memory) or MN-major, B likewise
__host__ __device__ constexpr uint32_t idesc(int n, bool a_mn, bool b_mn) {
    return umma::idesc(1, 128, n) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16);
}

// D (+)= A[tensor memory] B
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %5, %5, %5}, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"((uint32_t)acc), "r"(0u)
        : "memory");
}

__device__ __forceinline__ void tm_ld16(uint32_t addr, float (&v)[16]) {
    uint32_t u[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(addr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ void tm_st8(uint32_t addr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 consecutive floats of shared memory (16-byte aligned, the same for the warp)
__device__ __forceinline__ void get16(const float *p, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 f = reinterpret_cast<const float4 *>(p)[i];
        v[4 * i] = f.x;
        v[4 * i + 1] = f.y;
        v[4 * i + 2] = f.z;
        v[4 * i + 3] = f.w;
    }
}

// 16 floats (consecutive K elements of a lane, one K step) as N parts of
// 8 columns: the high and middle ones side by side at `at`, which is where an
// accumulator of the same 16 columns lies, the low one at `lo`
template <int N>
__device__ __forceinline__ void tm_parts16(uint32_t at, uint32_t lo, const float (&v)[16]) {
    uint32_t p[N][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t s[N];
        split<N>(v[2 * i], v[2 * i + 1], s);
#pragma unroll
        for (int j = 0; j < N; ++j) p[j][i] = s[j];
    }
    tm_st8(at, p[0]);
    if constexpr (N > 1) tm_st8(at + 8, p[1]);
    if constexpr (N > 2) tm_st8(lo, p[2]);
}
__device__ __forceinline__ void tm_split16(uint32_t at, uint32_t lo, const float (&v)[16]) {
    tm_parts16<3>(at, lo, v);
}

// 16 bytes to shared memory, zeros where `in` is false
__device__ __forceinline__ void cp16(void *dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(saddr(dst)), "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}

// `rows` rows (zeros up to 64) of dk elements (zeros up to DKT) into the parts'
// images, `part` bytes apart, column groups `group` bytes apart, from row 0 of
// dst. Warp w of nw takes every nw-th group of 8 rows, 4 column groups at a
// time. bf16 goes asynchronously (umma::cp_async_wait_all), the others by
// registers.
template <typename T, int DKT>
__device__ __forceinline__ void load_image(unsigned char *dst, int part, int group, const T *src, long long stride,
                                           int rows, int dk, int w, int nw) {
    constexpr int NB = Parts<T>::n;
    const int r = threadIdx.x & 7, cl = (threadIdx.x & 31) >> 3;
    src += r * stride + 8 * cl;
    dst += r * 16 + cl * group;
    for (int rg = w; rg < kC / 8; rg += nw) {
        const T *p = src + 8 * rg * stride;
        unsigned char *d = dst + rg * 128;
        const bool row = 8 * rg + r < rows;
        if constexpr (NB == 1) {
#pragma unroll
            for (int n = 0; n < DKT / 32; ++n) {
                const bool in = row && 8 * cl + 32 * n < dk;
                cp16(d + 4 * n * group, in ? p + 32 * n : src, in);
            }
        } else {
            uint4 v[DKT / 32][NB];
#pragma unroll
            for (int n = 0; n < DKT / 32; ++n) {
#pragma unroll
                for (int i = 0; i < NB; ++i) v[n][i] = make_uint4(0, 0, 0, 0);
                if (row && 8 * cl + 32 * n < dk) load_parts(p + 32 * n, v[n]);
            }
#pragma unroll
            for (int n = 0; n < DKT / 32; ++n)
#pragma unroll
                for (int i = 0; i < NB; ++i) *reinterpret_cast<uint4 *>(d + i * part + 4 * n * group) = v[n][i];
        }
    }
}

// Waits that run out. A wait may run out for some lanes of a warp only, but
// tensor-memory loads, elect and barriers need them all: so a lane notes it and
// goes on, over what is not there, and whole warps ask all_ok once a chunk,
// where they wait anyway, and leave together. A warp hands a stage back only
// behind that, when it has seen it filled: no copy is started over one under
// way. (Asking behind every wait cost 1 to 3% of the chains.)
__device__ __forceinline__ void try_wait(bool &ok, uint64_t *m, uint32_t parity) {
    ok = umma::mbar_wait(m, parity, kSpinLimit) && ok;
}
__device__ __forceinline__ bool all_ok(bool ok) { return __all_sync(0xffffffffu, ok); }

// `count` copies went to `stages` stages in turn: the parity of the last one's
// phase in stage i, -1 where there is none
__host__ __device__ constexpr int last_parity(int count, int stages, int i) {
    return count > i ? (count - 1 - i) / stages & 1 : -1;
}
// Waits for the last copies of a block (its readers have, unless a wait ran
// out), by the threads that issued them.
__device__ __forceinline__ void drain_copies(uint64_t *full, int count, int stages) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (int i = 0; i < stages; ++i) {
        const int parity = last_parity(count, stages, i);
        if (parity >= 0) umma::mbar_wait(full + i, parity, kDrainLimit);
    }
}

__device__ __forceinline__ void mbar_arrive(uint64_t *m) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(m)) : "memory");
}
// bytes that copies will bring in the current phase; the caller has not arrived yet
__device__ __forceinline__ void mbar_expect(uint64_t *m, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(saddr(m)), "r"(bytes) : "memory");
}
// bytes a multiple of 16, both addresses 16-byte aligned
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *m) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     saddr(dst)),
                 "l"(src), "r"(bytes), "r"(saddr(m))
                 : "memory");
}

__device__ __forceinline__ void bulk_prefetch(const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// `rows` rows of dv elements (zeros up to 64 rows) to consecutive places of
// dst, by thread t of nt; done when m has this thread's arrival (one of those
// it was initialised with). (Bulk copies of single rows take ~70 cycles each
// to issue, four times as long in all.)
template <typename T>
__device__ __forceinline__ void load_rows(unsigned char *dst, const T *src, long long stride, int rows, int dv, int t,
                                          int nt, uint64_t *m) {
    constexpr int E = 16 / (int)sizeof(T);
    const int per = dv / E, step = nt / per, r0 = t / per, c = t - r0 * per;   // per <= 32 <= nt
    if (r0 < step) {
        const T *p = src + r0 * stride + c * E;
        for (int r = r0; r < kC; r += step, p += step * stride) cp16(dst + (r * per + c) * 16, r < rows ? p : src, r < rows);
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(saddr(m)) : "memory");
}

// one lane of a converged warp; with warp-uniform operands the tensor-core
// instructions behind it issue back to back (a product of N columns every N / 2
// cycles; behind a test of the lane number they took up to 280)
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
template <typename V>
__device__ __forceinline__ V uniform(V v) { return __shfl_sync(0xffffffffu, v, 0); }

// the workspace: units of (slot, value head), then the images of [K; Q] of (slot, key head)
template <typename T, int DKT>
__host__ __device__ constexpr int kq_bytes() { return Parts<T>::n * 2 * kC * DKT * 2; }

// ----------------------------------------------------- the two chains ----
// warps 0-7: element-wise steps; 8: products; 9-11: loads
constexpr int kEpiWarps = 8, kLoadWarps = 3, kThreads = (kEpiWarps + 1 + kLoadWarps) * 32;

// parts of [K; Q], 128 rows; then T and PT and factors, V as it is
template <typename T, int DKT>
struct Stage {
    static constexpr int NB = Parts<T>::n;
    static constexpr int kImg = 2 * kC * DKT * 2, kTp = NB * kImg, kV = kTp + kUnitBytes;
    static __host__ __device__ int bytes(int dv) { return kV + kC * dv * (int)sizeof(T); }
    static __host__ __device__ int count(int dv) { return 2 * bytes(dv) + 256 <= 232448 ? 2 : 1; }
};

// One chunk's stage, by the loading threads (lt): images and unit as they lie
// in the workspace, and 64 rows of V or dO; full when m has kLoadWarps * 32 + 1
// arrivals and the copies' bytes.
template <typename T, int DKT>
__device__ __forceinline__ void load_stage(unsigned char *sp, const unsigned char *image, const unsigned char *unit,
                                           const T *rows, long long stride, int left, int dv, int lt, uint64_t *m) {
    using L = Stage<T, DKT>;
    if (lt == 0) {
        mbar_expect(m, kUnitBytes + L::kTp);
        bulk_load(sp, image, L::kTp, m);
        bulk_load(sp + L::kTp, unit, kUnitBytes, m);
        mbar_arrive(m);
    }
    load_rows<T>(sp + L::kV, rows, stride, left < kC ? left : kC, dv, lt, kLoadWarps * 32, m);
}
// the same on its way to L2
template <typename T, int DKT>
__device__ __forceinline__ void prefetch_stage(const unsigned char *image, const unsigned char *unit, const T *rows,
                                               long long stride, int left, int dv, int lt) {
    if (lt < kC && lt < left) {
        const char *p = (const char *)(rows + lt * stride);
        for (int i = 0; i < dv * (int)sizeof(T); i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i));
    }
    if (lt == kC) {
        bulk_prefetch(unit, kUnitBytes);
        bulk_prefetch(image, Stage<T, DKT>::kTp);
    }
}

// 16 tokens of this lane's channel to o, `row` elements apart, the first n of
// them. 16-bit types: neighbouring lanes swap so that each stores two channels
// of every other token in one word (dv is even: both channels are there or not).
template <typename T>
__device__ __forceinline__ void store16(T *o, long long row, const float (&x)[16], int lane, bool vin, int n) {
    if constexpr (sizeof(T) == 4) {
        if (vin) {
            if (n >= 16) {
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j * row] = x[j];
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < n) o[j * row] = x[j];
            }
        }
    } else {
        const bool odd = lane & 1;
        Pack<T, 2> w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float other = __shfl_xor_sync(0xffffffffu, odd ? x[2 * j] : x[2 * j + 1], 1);
            w[j].v[0] = from_f<T>(odd ? other : x[2 * j]);
            w[j].v[1] = from_f<T>(odd ? x[2 * j + 1] : other);
        }
        if (odd) {   // the odd lane has the second token of each pair
            o += row - 1;
            --n;
        }
        if (vin) {
            if (n >= 15) {
#pragma unroll
                for (int j = 0; j < 8; ++j) *reinterpret_cast<Pack<T, 2> *>(o + 2 * j * row) = w[j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (2 * j < n) *reinterpret_cast<Pack<T, 2> *>(o + 2 * j * row) = w[j];
            }
        }
    }
}

// What the gradient kernel reads: states as [dk / 4][dv][4] (a lane of the
// chains, one v, stores 4 of its dk; a warp 512 bytes in a row), E and dR as
// [dv / 8][64][8], 8 consecutive elements of a row and the rows side by side.
template <int HC>
__device__ __forceinline__ void store_state(float *p, const float (&S)[HC], int h, int v, int dk, int dv) {
#pragma unroll
    for (int i = 0; i < HC; i += 4)
        if (h * HC + i < dk)
            *reinterpret_cast<float4 *>(p + ((size_t)((h * HC + i) / 4) * dv + v) * 4) =
                make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
}
__device__ __forceinline__ void store_tokens(float *p, const float (&x)[16], int j0, int v) {
    p += ((v >> 3) * kC + j0) * 8 + (v & 7);
#pragma unroll
    for (int j = 0; j < 16; ++j) p[8 * j] = x[j];
}

}  // namespace delta
}  // namespace s4
