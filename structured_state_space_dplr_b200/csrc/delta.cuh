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
// of parts whose order is at least 2^-16 are summed, so that results are as
// good as float's, whatever their scale; a bf16 input is one part, a half two.
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
constexpr int kTpImage = 2 * kC * kC * 2;      // 16 KB: one part of [T; PT], 128 rows x 64 columns
constexpr int kTpBytes = 3 * kTpImage;
constexpr int kFacBytes = 2 * kC * 4;          // e^G and beta e^(G_C - G)
constexpr int kUnitBytes = kTpBytes + kFacBytes;   // workspace of one chunk and value head
constexpr uint32_t kSpinLimit = 1u << 22;

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
__host__ __device__ inline long long slots(long long tokens, int n) { return tokens / kC + n; }

// ---------------------------------------------------------------- split ----
__device__ __forceinline__ float lo_f(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float hi_f(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// a and b as N bf16 parts each, a in the low halves; each part is what the
// ones before it leave, rounded to nearest
template <int N>
__device__ __forceinline__ void split(float a, float b, uint32_t (&p)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        p[i] = pack2(a, b);
        a -= lo_f(p[i]);
        b -= hi_f(p[i]);
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

// 16 floats (consecutive K elements of a lane) as three parts of 8 columns each
__device__ __forceinline__ void tm_split16(uint32_t hi, uint32_t mid, uint32_t lo, const float (&v)[16]) {
    uint32_t p[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t s[3];
        split<3>(v[2 * i], v[2 * i + 1], s);
        p[0][i] = s[0];
        p[1][i] = s[1];
        p[2][i] = s[2];
    }
    tm_st8(hi, p[0]);
    tm_st8(mid, p[1]);
    tm_st8(lo, p[2]);
}

__device__ __forceinline__ void mbar_arrive(uint64_t *m) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(m)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t *m, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(m)), "r"(bytes) : "memory");
}
// bytes a multiple of 16, both addresses 16-byte aligned
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *m) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     saddr(dst)),
                 "l"(src), "r"(bytes), "r"(saddr(m))
                 : "memory");
}

}  // namespace delta
}  // namespace s4
