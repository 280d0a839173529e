// delta_prep.cu -- the part of the chunked gated delta rule that does not
// depend on the state: for every chunk and value head the images of
// T = (I + A D_b)^-1 and PT = P D_b T and the gates' factors.
//
// One block per chunk and value head, 128 threads. [K; Q] K^T is one M = 128
// product (rows 0-63 give A, rows 64-127 give P); a thread owns a row of the
// accumulator. T is inverted in float: the two 32 x 32 diagonal blocks by
// forward substitution, a column a thread, then T21 = -T22 A21 T11. PT is a
// second product with P as operand in tensor memory.
#include "delta.cuh"
#include "s4dplr.h"

namespace s4 {
namespace {

using namespace delta;

constexpr int kLd = kC + 4;   // row stride of the float matrices: 16-byte rows, shifted banks

template <typename T, int DKT>
struct PrepSmem {
    static constexpr int kKq = Parts<T>::n * 2 * kC * DKT * 2;   // images of [K; Q], 128 rows
    static constexpr int kTImg = kC * kC * 2;                    // one part of T, 64 x 64
    static constexpr int kFloat = 2 * kC * kLd * 4;              // A D_b, T
    static constexpr int kImg = kKq > 3 * kTImg ? kKq : 3 * kTImg;   // T's images take the place of K's and Q's
    static constexpr int kBytes = kImg + kFloat + kC * 8 + 2 * kC * 4 + 64;
};

template <typename T, int DKT>
__global__ void __launch_bounds__(128) k_delta_prep(DeltaArgs a, unsigned char *ws, unsigned *flags) {
    using L = PrepSmem<T, DKT>;
    constexpr int NB = Parts<T>::n;
    extern __shared__ __align__(1024) unsigned char smem[];
    float *As = reinterpret_cast<float *>(smem + L::kImg), *Ts = As + kC * kLd;
    double *Gs = reinterpret_cast<double *>(Ts + kC * kLd);
    float *gs = reinterpret_cast<float *>(Gs + kC), *bs = gs + kC;
    uint64_t *bar = reinterpret_cast<uint64_t *>(bs + kC);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const long long slot = blockIdx.x / a.hv;
    const int hv = blockIdx.x % a.hv, hk = hv / (a.hv / a.hk);
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
    if (c0 < 0 || c0 >= sq.len) return;   // a slot no chunk uses
    const int rows = sq.len - c0 < kC ? (int)(sq.len - c0) : kC;
    const long long tok = sq.tok0 + c0;

    if (warp == 0) umma::tmem_alloc(tslot, 256);
    if (tid == 0) {
        umma::mbar_init(bar, 1);
        umma::fence_mbar_init();
    }
    {   // [K; Q] into the images: a warp takes 8 rows x 4 column groups at a time
        constexpr int kUnits = 16 * (DKT / 32);
        for (int u = warp; u < kUnits; u += 4) {
            const int r = (u / (DKT / 32)) * 8 + (lane & 7), cg = (u % (DKT / 32)) * 4 + (lane >> 3);
            const int row = r & (kC - 1);
            uint4 p[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) p[i] = make_uint4(0, 0, 0, 0);
            if (row < rows && 8 * cg < a.dk) {
                const T *src = r < kC ? (const T *)a.k + (tok + row) * a.sk : (const T *)a.q + (tok + row) * a.sq;
                load_parts(src + (long long)hk * a.dk + 8 * cg, p);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i)
                *reinterpret_cast<uint4 *>(smem + i * (2 * kC * DKT * 2) + (r >> 3) * 128 + cg * 2048 + (r & 7) * 16) =
                    p[i];
        }
    }
    if (warp == 1) {   // running sums of g in double: differences of large sums keep float's accuracy
        const int j = 2 * lane;
        const long long at = tok * a.hv + hv;
        float g0 = j < rows ? __ldg(a.g + at + (long long)j * a.hv) : 0.0f;
        float g1 = j + 1 < rows ? __ldg(a.g + at + (long long)(j + 1) * a.hv) : 0.0f;
        // exp(-1e5) is 0 as exp(-inf) is, and differences stay numbers
        g0 = g0 < -1e5f ? -1e5f : g0;
        g1 = g1 < -1e5f ? -1e5f : g1;
        double x = (double)g0 + (double)g1, y = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        Gs[j] = y - (double)g1;
        Gs[j + 1] = y;
        bs[j] = j < rows ? __ldg(a.beta + at + (long long)j * a.hv) : 0.0f;
        bs[j + 1] = j + 1 < rows ? __ldg(a.beta + at + (long long)(j + 1) * a.hv) : 0.0f;
    }
    umma::fence_proxy_async();
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tm = *tslot;
    uint32_t phase = 0;
    bool ok = true;
    if (tid == 0) {
        const uint32_t base = saddr(smem);
        bool acc = false;
#pragma unroll
        for (int o = 2; o >= 0; --o)   // parts' products, the smallest first
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int j = o - i;
                if (j < 0 || j >= NB) continue;
                for (int ks = 0; ks < DKT / 16; ++ks) {
                    umma::mma_bf16(tm, desc_k(base + i * (2 * kC * DKT * 2) + ks * 4096, 2048, 128),
                                   desc_k(base + j * (2 * kC * DKT * 2) + ks * 4096, 2048, 128), idesc(kC, false, false),
                                   acc);
                    acc = true;
                }
            }
        umma::commit(bar);
    }
    ok = umma::mbar_wait(bar, phase, kSpinLimit);
    phase ^= 1;
    umma::fence_after_sync();
    const uint32_t mine = tm + ((uint32_t)(warp * 32) << 16);
    const int i = tid & (kC - 1);   // this thread's row of A or of P
    {
        const double Gi = Gs[i];
#pragma unroll
        for (int c = 0; c < kC; c += 16) {
            float d[16];
            tm_ld16(mine + c, d);
            if (tid < kC) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    d[j] = c + j < i ? d[j] * expf((float)(Gi - Gs[c + j])) * bs[c + j] : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<float4 *>(As + i * kLd + c + j) = make_float4(d[j], d[j + 1], d[j + 2], d[j + 3]);
#pragma unroll
                for (int j = 0; j < 16; ++j) d[j] = 0.0f;   // rows 0-63 of the second product's operand are not used
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    d[j] = c + j <= i ? d[j] * (a.scale * bs[c + j]) * expf((float)(Gi - Gs[c + j])) : 0.0f;
            }
            tm_split16(mine + 64 + c / 2, mine + 96 + c / 2, mine + 128 + c / 2, d);
        }
        tm_wait_st();
        if (tid >= kC) {
            unsigned char *fac = ws + (size_t)blockIdx.x * kUnitBytes + kTpBytes;
            reinterpret_cast<float *>(fac)[i] = expf((float)Gi);
            reinterpret_cast<float *>(fac)[kC + i] = bs[i] * expf((float)(Gs[kC - 1] - Gi));
        }
    }
    __syncthreads();
    // T11 and T22 by columns: x_r = [r = c] - sum_{j < r} A_rj x_j
    if (warp < 2) {
        const int o = 32 * warp;
        float x[32];
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            float acc[4] = {r == lane ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < r; j += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(As + (o + r) * kLd + o + j);
                acc[0] = fmaf(-v.x, x[j], acc[0]);
                if (j + 1 < r) acc[1] = fmaf(-v.y, x[j + 1], acc[1]);
                if (j + 2 < r) acc[2] = fmaf(-v.z, x[j + 2], acc[2]);
                if (j + 3 < r) acc[3] = fmaf(-v.w, x[j + 3], acc[3]);
            }
            x[r] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            Ts[(o + r) * kLd + o + lane] = x[r];
        }
    } else if (warp == 2) {   // T12 = 0
#pragma unroll
        for (int r = 0; r < 32; ++r) Ts[r * kLd + 32 + lane] = 0.0f;
    }
    __syncthreads();
    {   // T21 = -T22 (A21 T11): row and 8 columns of it a thread
        const int r = tid >> 2, c = (tid & 3) * 8;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.0f;
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
            const float v = As[(32 + r) * kLd + k];
            const float4 p = *reinterpret_cast<const float4 *>(Ts + k * kLd + c);
            const float4 q = *reinterpret_cast<const float4 *>(Ts + k * kLd + c + 4);
            y[0] = fmaf(v, p.x, y[0]);
            y[1] = fmaf(v, p.y, y[1]);
            y[2] = fmaf(v, p.z, y[2]);
            y[3] = fmaf(v, p.w, y[3]);
            y[4] = fmaf(v, q.x, y[4]);
            y[5] = fmaf(v, q.y, y[5]);
            y[6] = fmaf(v, q.z, y[6]);
            y[7] = fmaf(v, q.w, y[7]);
        }
        // the rows 0-31 of A are used up: A21 T11 goes there
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; j += 4)
            *reinterpret_cast<float4 *>(As + r * kLd + c + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.0f;
#pragma unroll 8
        for (int k = 0; k < 32; ++k) {
            const float v = -Ts[(32 + r) * kLd + 32 + k];
            const float4 p = *reinterpret_cast<const float4 *>(As + k * kLd + c);
            const float4 q = *reinterpret_cast<const float4 *>(As + k * kLd + c + 4);
            y[0] = fmaf(v, p.x, y[0]);
            y[1] = fmaf(v, p.y, y[1]);
            y[2] = fmaf(v, p.z, y[2]);
            y[3] = fmaf(v, p.w, y[3]);
            y[4] = fmaf(v, q.x, y[4]);
            y[5] = fmaf(v, q.y, y[5]);
            y[6] = fmaf(v, q.z, y[6]);
            y[7] = fmaf(v, q.w, y[7]);
        }
#pragma unroll
        for (int j = 0; j < 8; j += 4)
            *reinterpret_cast<float4 *>(Ts + (32 + r) * kLd + c + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
    }
    __syncthreads();
    unsigned char *out = ws + (size_t)blockIdx.x * kUnitBytes;
    {   // T's parts: into shared memory as operand (64 rows) and to the workspace (rows 0-63 of [T; PT])
        const int r = tid & 63;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int cg = (tid >> 6) * 4 + n;
            uint32_t w[4][3];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                split<3>(Ts[r * kLd + 8 * cg + 2 * j], Ts[r * kLd + 8 * cg + 2 * j + 1], w[j]);
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const uint4 v = make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
                *reinterpret_cast<uint4 *>(smem + q * L::kTImg + (r >> 3) * 128 + cg * 1024 + (r & 7) * 16) = v;
                *reinterpret_cast<uint4 *>(out + q * kTpImage + (r >> 3) * 128 + cg * 2048 + (r & 7) * 16) = v;
            }
        }
    }
    umma::fence_proxy_async();
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    if (tid == 0) {   // PT = P' T: K runs over T's rows
        const uint32_t base = saddr(smem);
        bool acc = false;
#pragma unroll
        for (int o = 2; o >= 0; --o)
#pragma unroll
            for (int p = 0; p <= o; ++p)
                for (int ks = 0; ks < kC / 16; ++ks) {
                    mma_ts(tm, tm + 64 + 32 * p + 8 * ks, desc_mn(base + (o - p) * L::kTImg + ks * 256, 128, 1024),
                           idesc(kC, false, true), acc);
                    acc = true;
                }
        umma::commit(bar);
    }
    ok = umma::mbar_wait(bar, phase, kSpinLimit) && ok;
    umma::fence_after_sync();
    if (tid >= kC) {
#pragma unroll
        for (int c = 0; c < kC; c += 16) {
            float d[16];
            tm_ld16(mine + c, d);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[4][3];
#pragma unroll
                for (int j = 0; j < 4; ++j) split<3>(d[8 * h + 2 * j], d[8 * h + 2 * j + 1], w[j]);
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    *reinterpret_cast<uint4 *>(out + q * kTpImage + (8 + (i >> 3)) * 128 + (c / 8 + h) * 2048 +
                                               (i & 7) * 16) = make_uint4(w[0][q], w[1][q], w[2][q], w[3][q]);
            }
        }
    }
    if (!ok && flags && tid == 0) atomicOr(flags, S4_FLAG_TIMEOUT);
    umma::fence_before_sync();
    __syncthreads();
    if (warp == 0) umma::tmem_dealloc(tm, 256);
}

template <typename T, int DKT>
cudaError_t run(const DeltaArgs &a, void *ws, unsigned *flags, cudaStream_t st) {
    constexpr int smem = PrepSmem<T, DKT>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(k_delta_prep<T, DKT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const long long grid = slots(a.tokens, a.n) * a.hv;
    k_delta_prep<T, DKT><<<(unsigned)grid, 128, smem, st>>>(a, (unsigned char *)ws, flags);
    return cudaGetLastError();
}

}  // namespace

size_t delta_unit_bytes() { return delta::kUnitBytes; }

cudaError_t launch_delta_prep(int dtype, const DeltaArgs &a, void *ws, unsigned *flags, cudaStream_t st) {
    const bool wide = a.dk > 64;
    if (dtype == S4_BF16)
        return wide ? run<__nv_bfloat16, 128>(a, ws, flags, st) : run<__nv_bfloat16, 64>(a, ws, flags, st);
    if (dtype == S4_F16) return wide ? run<__half, 128>(a, ws, flags, st) : run<__half, 64>(a, ws, flags, st);
    return wide ? run<float, 128>(a, ws, flags, st) : run<float, 64>(a, ws, flags, st);
}

}  // namespace s4
