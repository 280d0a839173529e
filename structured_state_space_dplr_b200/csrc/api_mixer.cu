// api_mixer.cu -- the extern "C" entry points of the token-major operators:
// layer norm over rows, the backward of both layer norms, and the gated delta
// rule. Arguments are checked on the host before anything is launched;
// nothing here allocates device memory.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "launch.h"
#include "s4dplr.h"

namespace {

s4_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return S4_OK;
    s4::record_cuda_error(e);
    return S4_ERR_CUDA;
}

// one buffer of a call: address, bytes, whether the call writes it (null and empty buffers overlap nothing)
struct Buf {
    const void *p;
    double bytes;
    bool out;
};

bool overlapping(std::initializer_list<Buf> bufs) {
    for (const Buf *a = bufs.begin(); a != bufs.end(); ++a)
        for (const Buf *b = a + 1; b != bufs.end(); ++b) {
            if (!(a->out || b->out) || !a->p || !b->p || a->bytes == 0 || b->bytes == 0) continue;
            const double x = (double)(uintptr_t)a->p, y = (double)(uintptr_t)b->p;
            // addresses are below 2^53: exact as doubles
            if (x < y + b->bytes && y < x + a->bytes) return true;
        }
    return false;
}

bool aligned(size_t a, std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if ((uintptr_t)p % a) return false;
    return true;
}

bool any_null(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!p) return true;
    return false;
}

bool dtype_ok(int t) { return t == S4_F32 || t == S4_BF16 || t == S4_F16; }
size_t dtype_size(int t) { return t == S4_F32 ? 4 : 2; }

s4_status rows_checks(int dtype, long long rows, int D) {
    if (!dtype_ok(dtype) || rows < 0 || D < 1) return S4_ERR_INVALID_ARG;
    if (D > S4_MAX_BLOCK_H || rows > 0x7fffffffLL) return S4_ERR_UNSUPPORTED;
    return S4_OK;
}

// sizes of the gated delta rule
s4_status delta_sizes(int dtype, int Bt, int Hk, int Hv, int Dk, int Dv) {
    if (!dtype_ok(dtype) || Bt < 1 || Hk < 1 || Hv < 1 || Dk < 1 || Dv < 1 || Hv % Hk) return S4_ERR_INVALID_ARG;
    if (Dk % 8 || Dv % 8 || Dk > S4_MAX_DELTA_D || Dv > S4_MAX_DELTA_D) return S4_ERR_UNSUPPORTED;
    if ((double)Bt * Hv > 2147483647.0) return S4_ERR_UNSUPPORTED;
    return S4_OK;
}

bool strides_ok(int dtype, int Hk, int Hv, int Dk, int Dv, long long sq, long long sk, long long sv) {
    const long long unit = 16 / (long long)dtype_size(dtype);
    return sq >= (long long)Hk * Dk && sk >= (long long)Hk * Dk && sv >= (long long)Hv * Dv && sq % unit == 0 &&
           sk % unit == 0 && sv % unit == 0;
}

// bytes from the first to the last element of `tokens` rows of `row` elements, `stride` apart
double span(int dtype, double tokens, long long stride, long long row) {
    return tokens < 1 ? 0.0 : ((tokens - 1) * (double)stride + (double)row) * (double)dtype_size(dtype);
}

// the workspace of the chunked form: units of T and PT and factors, then (keep)
// the states before the chunks, E, the states' gradients behind the chunks and
// dR, then the segments' summaries
struct DeltaWork {
    size_t state, rows, prep, sums, total;   // bytes of one kind
    int seg;
};
DeltaWork delta_work(int dtype, bool packed, int Bt, long long tokens, int Hk, int Hv, int Dk, int Dv, int keep) {
    DeltaWork w;
    const long long units = (tokens / 64 + Bt) * (long long)Hv;
    w.prep = s4::delta_prep_bytes(dtype, tokens, Bt, Hk, Hv, Dk);
    w.state = keep ? (size_t)units * Dk * Dv * 4 : 0;
    w.rows = keep ? (size_t)units * 64 * Dv * 4 : 0;
    long long segments;
    w.seg = s4::delta_segment(tokens, Bt, Hv, packed, &segments);
    w.sums = s4::delta_segment_bytes(segments, Hv, Dk, Dv, keep);
    w.total = w.prep + 2 * w.state + 2 * w.rows + w.sums;
    return w;
}

// sizes of the chunked form; `tokens` in all, packed (cu) or Bt times the same number
s4_status chunk_sizes(int dtype, bool packed, int Bt, long long tokens, int Hk, int Hv, int Dk, int Dv) {
    s4_status s = delta_sizes(dtype, Bt, Hk, Hv, Dk, Dv);
    if (s != S4_OK) return s;
    if (tokens < 0 || (!packed && tokens % Bt)) return S4_ERR_INVALID_ARG;
    if (tokens > 0x7fffffffLL || (double)(tokens / 64 + Bt) * Hv > 2147483647.0) return S4_ERR_UNSUPPORTED;
    return S4_OK;
}

}  // namespace

extern "C" {

s4_status s4_layernorm(s4_dtype dtype, const void *x, const float *gamma, const float *beta, float eps,
                       long long rows, int D, void *z, float *mean, float *rstd, cudaStream_t stream) {
    s4_status s = rows_checks(dtype, rows, D);
    if (s != S4_OK) return s;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return S4_ERR_INVALID_ARG;
    if (rows == 0) return S4_OK;
    if (any_null({x, gamma, beta, z, mean, rstd})) return S4_ERR_INVALID_ARG;
    const size_t e = dtype_size(dtype);
    if (!aligned(e, {x, z}) || !aligned(4, {gamma, beta, mean, rstd})) return S4_ERR_INVALID_ARG;
    const double n = (double)rows * D * e, r = 4.0 * rows, w = 4.0 * D;
    // in place (z = x) is allowed: a row is read whole before it is written
    if (overlapping({{z == x ? nullptr : x, n, false}, {gamma, w, false}, {beta, w, false}, {z, n, true},
                     {mean, r, true}, {rstd, r, true}}))
        return S4_ERR_INVALID_ARG;
    return cuda_status(s4::launch_layernorm_rows(dtype, x, gamma, beta, eps, rows, D, z, mean, rstd, stream));
}

s4_status s4_layernorm_backward_workspace_size(int D, size_t *bytes) {
    if (!bytes || D < 1) return S4_ERR_INVALID_ARG;
    if (D > S4_MAX_BLOCK_H) return S4_ERR_UNSUPPORTED;
    *bytes = s4::norm_backward_workspace_bytes(D);
    return S4_OK;
}

s4_status s4_layernorm_backward(s4_dtype dtype, const void *dz, const void *x, const float *gamma, const float *mean,
                                const float *rstd, long long rows, int D, void *dx, float *dgamma, float *dbeta,
                                void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    s4_status s = rows_checks(dtype, rows, D);
    if (s != S4_OK) return s;
    if (any_null({gamma, dgamma, dbeta})) return S4_ERR_INVALID_ARG;
    if (rows > 0 && any_null({dz, x, mean, rstd, dx})) return S4_ERR_INVALID_ARG;
    const size_t e = dtype_size(dtype);
    if (!aligned(e, {dz, x, dx}) || !aligned(4, {gamma, mean, rstd, dgamma, dbeta})) return S4_ERR_INVALID_ARG;
    if (!workspace || !aligned(256, {workspace}) || workspace_bytes < s4::norm_backward_workspace_bytes(D))
        return S4_ERR_WORKSPACE;
    const double n = (double)rows * D * e, r = 4.0 * rows, w = 4.0 * D;
    // in place (dx = dz) is allowed: a row is read whole before it is written
    if (overlapping({{dx == dz ? nullptr : dz, n, false}, {x, n, false}, {gamma, w, false}, {mean, r, false},
                     {rstd, r, false}, {dx, n, true}, {dgamma, w, true}, {dbeta, w, true},
                     {workspace, (double)workspace_bytes, true}}))
        return S4_ERR_INVALID_ARG;
    return cuda_status(s4::launch_layernorm_rows_backward(dtype, dz, x, gamma, mean, rstd, rows, D, dx, dgamma, dbeta,
                                                          workspace, stream));
}

s4_status s4_layernorm_channels_backward(const float *dz, const float *x, const float *gamma, float eps, int Bt,
                                         int H, int L, float *dx, float *dgamma, float *dbeta, void *workspace,
                                         size_t workspace_bytes, cudaStream_t stream) {
    if (any_null({dz, x, gamma, dx, dgamma, dbeta}) || Bt < 1 || H < 1 || H > S4_MAX_BLOCK_H || !(eps > 0.0f) ||
        !std::isfinite(eps))
        return S4_ERR_INVALID_ARG;
    if (L < S4_MIN_L || L > S4_MAX_L || (L & (L - 1))) return S4_ERR_UNSUPPORTED;
    if ((double)Bt * H * L >= 1099511627776.0) return S4_ERR_INVALID_ARG;   // 2^40
    if (!aligned(16, {dz, x, dx}) || !aligned(4, {gamma, dgamma, dbeta})) return S4_ERR_INVALID_ARG;
    if (!workspace || !aligned(256, {workspace}) || workspace_bytes < s4::norm_backward_workspace_bytes(H))
        return S4_ERR_WORKSPACE;
    const double n = 4.0 * Bt * H * L, w = 4.0 * H;
    if (overlapping({{dz, n, false}, {x, n, false}, {gamma, w, false}, {dx, n, true}, {dgamma, w, true},
                     {dbeta, w, true}, {workspace, (double)workspace_bytes, true}}))
        return S4_ERR_INVALID_ARG;
    return cuda_status(s4::launch_layernorm_channels_backward(dz, x, gamma, eps, Bt, H, L, dx, dgamma, dbeta,
                                                              workspace, stream));
}

s4_status s4_gated_delta_scan(s4_dtype dtype, const void *q, long long q_stride, const void *k, long long k_stride,
                              const void *v, long long v_stride, const float *g, const float *beta, float scale,
                              float *state, int Bt, int T, int Hk, int Hv, int Dk, int Dv, void *o,
                              cudaStream_t stream) {
    s4_status s = delta_sizes(dtype, Bt, Hk, Hv, Dk, Dv);
    if (s != S4_OK) return s;
    if (T < 0 || !std::isfinite(scale) || !strides_ok(dtype, Hk, Hv, Dk, Dv, q_stride, k_stride, v_stride))
        return S4_ERR_INVALID_ARG;
    if (T == 0) return S4_OK;
    if (any_null({q, k, v, g, beta, state, o})) return S4_ERR_INVALID_ARG;
    if (!aligned(16, {q, k, v, o, state}) || !aligned(4, {g, beta})) return S4_ERR_INVALID_ARG;
    const double tok = (double)Bt * T, gate = tok * Hv * 4.0;
    if (overlapping({{q, span(dtype, tok, q_stride, (long long)Hk * Dk), false},
                     {k, span(dtype, tok, k_stride, (long long)Hk * Dk), false},
                     {v, span(dtype, tok, v_stride, (long long)Hv * Dv), false},
                     {g, gate, false},
                     {beta, gate, false},
                     {state, 4.0 * Bt * Hv * Dk * Dv, true},
                     {o, span(dtype, tok, (long long)Hv * Dv, (long long)Hv * Dv), true}}))
        return S4_ERR_INVALID_ARG;
    s4::DeltaArgs a{q, k, v, g, beta, o, Bt, Hk, Hv, Dk, Dv, q_stride, k_stride, v_stride, scale, nullptr, T, Bt * (long long)T, 0};
    return cuda_status(s4::launch_delta_scan(dtype, a, state, T, stream));
}

s4_status s4_gated_delta_workspace_size(s4_dtype dtype, int Bt, long long tokens, int Hk, int Hv, int Dk, int Dv,
                                        int keep, size_t *bytes) {
    if (!bytes) return S4_ERR_INVALID_ARG;
    s4_status s = chunk_sizes(dtype, true, Bt, tokens, Hk, Hv, Dk, Dv);
    if (s != S4_OK) return s;
    const size_t packed = delta_work(dtype, true, Bt, tokens, Hk, Hv, Dk, Dv, keep).total;
    const size_t equal = delta_work(dtype, false, Bt, tokens, Hk, Hv, Dk, Dv, keep).total;
    *bytes = packed > equal ? packed : equal;
    return S4_OK;
}

s4_status s4_gated_delta_forward(s4_dtype dtype, const void *q, long long q_stride, const void *k, long long k_stride,
                                 const void *v, long long v_stride, const float *g, const float *beta, float scale,
                                 const float *initial_state, const int *cu_seqlens, int Bt, long long tokens, int Hk,
                                 int Hv, int Dk, int Dv, void *o, float *final_state, int keep, void *workspace,
                                 size_t workspace_bytes, unsigned *d_flags, cudaStream_t stream) {
    s4_status s = chunk_sizes(dtype, cu_seqlens != nullptr, Bt, tokens, Hk, Hv, Dk, Dv);
    if (s != S4_OK) return s;
    if (!std::isfinite(scale) || !strides_ok(dtype, Hk, Hv, Dk, Dv, q_stride, k_stride, v_stride))
        return S4_ERR_INVALID_ARG;
    if (tokens > 0 && any_null({q, k, v, g, beta, o})) return S4_ERR_INVALID_ARG;
    if (!aligned(16, {q, k, v, o, initial_state, final_state}) || !aligned(4, {g, beta, cu_seqlens, d_flags}))
        return S4_ERR_INVALID_ARG;
    const DeltaWork w = delta_work(dtype, cu_seqlens != nullptr, Bt, tokens, Hk, Hv, Dk, Dv, keep);
    if (!workspace || !aligned(256, {workspace}) || workspace_bytes < w.total) return S4_ERR_WORKSPACE;
    const double tok = (double)tokens, gate = tok * Hv * 4.0, st = 4.0 * Bt * Hv * Dk * Dv;
    // final_state may be initial_state: a state is read before it is written
    if (overlapping({{q, span(dtype, tok, q_stride, (long long)Hk * Dk), false},
                     {k, span(dtype, tok, k_stride, (long long)Hk * Dk), false},
                     {v, span(dtype, tok, v_stride, (long long)Hv * Dv), false},
                     {g, gate, false},
                     {beta, gate, false},
                     {cu_seqlens, 4.0 * (Bt + 1.0), false},
                     {initial_state == final_state ? nullptr : initial_state, st, false},
                     {o, span(dtype, tok, (long long)Hv * Dv, (long long)Hv * Dv), true},
                     {final_state, st, true},
                     {d_flags, 4.0, true},
                     {workspace, (double)workspace_bytes, true}}))
        return S4_ERR_INVALID_ARG;
    s4::DeltaArgs a{q,  k,  v,        g,        beta,     o,     Bt,         Hk,                        Hv,    Dk,
                    Dv, q_stride, k_stride, v_stride, scale, cu_seqlens, cu_seqlens ? 0 : (int)(tokens / Bt), tokens,
                    w.seg};
    char *p = (char *)workspace;
    float *ks = keep ? (float *)(p + w.prep) : nullptr, *ke = keep ? (float *)(p + w.prep + w.state) : nullptr;
    if (tokens > 0) {
        s = cuda_status(s4::launch_delta_prep(dtype, a, workspace, d_flags, stream));
        if (s != S4_OK) return s;
    }
    return cuda_status(
        s4::launch_delta_forward(dtype, a, initial_state, final_state, workspace, ks, ke,
                                 p + w.prep + 2 * w.state + 2 * w.rows, d_flags, stream));
}

s4_status s4_gated_delta_backward(s4_dtype dtype, const float *g, const float *beta, float scale,
                                  const int *cu_seqlens, int Bt, long long tokens, int Hk, int Hv, int Dk, int Dv,
                                  const void *d_o, const float *d_final_state, void *dq, void *dk, void *dv,
                                  float *dg, float *dbeta, float *d_initial_state, void *workspace,
                                  size_t workspace_bytes, unsigned *d_flags, cudaStream_t stream) {
    s4_status s = chunk_sizes(dtype, cu_seqlens != nullptr, Bt, tokens, Hk, Hv, Dk, Dv);
    if (s != S4_OK) return s;
    if (!std::isfinite(scale)) return S4_ERR_INVALID_ARG;
    if (tokens > 0 && any_null({g, beta, d_o, dq, dk, dv, dg, dbeta})) return S4_ERR_INVALID_ARG;
    if (!aligned(16, {d_o, dq, dk, dv, d_final_state, d_initial_state}) ||
        !aligned(4, {g, beta, dg, dbeta, cu_seqlens, d_flags}))
        return S4_ERR_INVALID_ARG;
    const DeltaWork w = delta_work(dtype, cu_seqlens != nullptr, Bt, tokens, Hk, Hv, Dk, Dv, 1);
    if (!workspace || !aligned(256, {workspace}) || workspace_bytes < w.total) return S4_ERR_WORKSPACE;
    const double tok = (double)tokens, gate = tok * Hv * 4.0, st = 4.0 * Bt * Hv * Dk * Dv;
    const double nk = tok * Hk * Dk * dtype_size(dtype), nv = tok * Hv * Dv * dtype_size(dtype);
    // d_initial_state may be d_final_state: a state is read before it is written
    if (overlapping({{g, gate, false},
                     {beta, gate, false},
                     {cu_seqlens, 4.0 * (Bt + 1.0), false},
                     {d_o, nv, false},
                     {d_final_state == d_initial_state ? nullptr : d_final_state, st, false},
                     {dq, nk, true},
                     {dk, nk, true},
                     {dv, nv, true},
                     {dg, gate, true},
                     {dbeta, gate, true},
                     {d_initial_state, st, true},
                     {d_flags, 4.0, true},
                     {workspace, (double)workspace_bytes, true}}))
        return S4_ERR_INVALID_ARG;
    s4::DeltaArgs a{};
    a.g = g, a.beta = beta, a.n = Bt, a.hk = Hk, a.hv = Hv, a.dk = Dk, a.dv = Dv, a.scale = scale;
    a.cu = cu_seqlens, a.t = cu_seqlens ? 0 : (int)(tokens / Bt), a.tokens = tokens, a.seg = w.seg;
    char *p = (char *)workspace + w.prep;
    float *ks = (float *)p, *ke = (float *)(p + w.state), *kds = (float *)(p + w.state + w.rows),
          *kdr = (float *)(p + 2 * w.state + w.rows);
    s = cuda_status(s4::launch_delta_backward(dtype, a, d_o, d_final_state, d_initial_state, workspace, dv, kds, kdr,
                                              p + 2 * w.state + 2 * w.rows, d_flags, stream));
    if (s != S4_OK || tokens == 0) return s;
    return cuda_status(
        s4::launch_delta_gradient(dtype, a, d_o, workspace, ks, ke, kds, kdr, dq, dk, dg, dbeta, d_flags, stream));
}

}  // extern "C"
