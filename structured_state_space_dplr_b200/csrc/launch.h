// launch.h -- internal host-side launchers (one per kernel family).
#pragma once
#include <cuda_runtime.h>
#include <atomic>
#include <cstddef>
#include <mutex>

namespace s4 {

// A kernel's limit of dynamic shared memory per device, raised to the largest
// size asked for and never lowered: calls of different sizes share a kernel and
// may come from several host threads at once, so that the limit and the record
// of it change together, under the lock.
struct SmemLimit {
    static constexpr int kDevices = 64;
    std::atomic<size_t> set[kDevices] = {};
    std::mutex change;
    template <typename K>
    cudaError_t raise(K *kernel, size_t bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev >= kDevices) return cudaErrorInvalidDevice;
        if (set[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
        std::lock_guard<std::mutex> lock(change);
        if (set[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e == cudaSuccess) set[dev].store(bytes, std::memory_order_release);
        return e;
    }
};

// Blocks of a kernel that an SM holds, asked for once per block size, which
// sets the shared memory (the same on every device this library runs on).
// Threads that ask at the same time write the same number.
struct Resident {
    std::atomic<int> n[33] = {};   // by block size / 32
    template <typename K>
    int of(K *kernel, int block, size_t smem) {
        std::atomic<int> &r = n[block / 32];
        int b = r.load(std::memory_order_relaxed);
        if (b == 0) {
            if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, kernel, block, smem) != cudaSuccess || b < 1) b = 1;
            r.store(b, std::memory_order_relaxed);
        }
        return b;
    }
};

// remember a failing CUDA call for s4_last_cuda_error() (calling host thread)
void record_cuda_error(cudaError_t e);

// ---- spectral.cu: FFT convolution and inverse real FFT ----
// Cluster split used for the length-2L convolution transforms.
struct ConvGeom { int C; int lg; };
ConvGeom conv_geom(int L);
size_t conv_workspace_bytes(int H, int L);

// spectrum of K + D delta_0 (D may be null: no feed-through) into ws; with Ki
// (L > 8192 only) the spectrum of the complex signal K + i Ki instead
cudaError_t launch_kspec(const float *K, const float *D, int H, int L, void *ws, cudaStream_t st,
                         const float *Ki = nullptr);
// adjoint: the correlation with the same spectrum (conjugated), y[s] = sum_{t>=s} K[t-s] u[t] + D u[s]
cudaError_t launch_fftconv(const float *u, const void *ws, int Bt, int H, int L, float *y, cudaStream_t st,
                           bool adjoint = false);
// in place: K[H, L] holds the packed half spectrum on entry, the real kernel on exit
// ---- backward.cu ----
size_t corr_workspace_bytes(int H, int L);
cudaError_t launch_corr(const float *u, const float *dy, int Bt, int H, int L, float *dK, float *dD, void *ws,
                        cudaStream_t st);

// L > 16384 needs kgen_backward_workspace_bytes(H, L) of workspace (ws), else ws may be null
size_t kgen_backward_workspace_bytes(int H, int L);
cudaError_t launch_kgen_backward(const float2 *Lambda, const float2 *P, const float2 *Q, const float2 *B,
                                 const float2 *C, const float *log_dt, const float *dK, int H, int Nh, int L,
                                 float2 *dLambda, float2 *dP, float2 *dQ, float2 *dB, float2 *dC,
                                 float *dlog_dt, void *ws, cudaStream_t st);

cudaError_t launch_irfft_packed(float *K, int H, int L, cudaStream_t st);
// K holds the packed half spectrum (k_cauchy's output) on entry and the kernel
// on exit; ws receives the spectrum of K + D delta_0 as launch_kspec leaves it
// (L = 16384: one fused launch; other L: launch_irfft_packed + launch_kspec)
cudaError_t launch_kspec_from_half(float *K, const float *D, int H, int L, void *ws, cudaStream_t st);

// ---- quad.cu: L = 16384 (a cluster of two CTAs holding four ranks) ----
cudaError_t launch_kspec_l16k(const float *K, const float *D, int H, void *ws, cudaStream_t st, const float *Ki);
cudaError_t launch_fftconv_l16k(const float *u, const void *ws, int Bt, int H, float *y, bool adjoint,
                                cudaStream_t st);
cudaError_t launch_kspec_from_half_l16k(float *K, const float *D, int H, void *ws, cudaStream_t st);

// ---- kgen.cu: K and the convolution spectrum of K + D delta_0 in one launch
// (L <= 8192; longer L runs k_cauchy, then launch_kspec_from_half) ----
cudaError_t launch_kgen(const float2 *Lambda, const float2 *P, const float2 *Q, const float2 *B, const float2 *C,
                        const float *log_dt, const float *D, int H, int Nh, int L, float *K, void *ws,
                        unsigned *flags, cudaStream_t st);

// ---- cauchy.cu ----
cudaError_t launch_cauchy(const float2 *Lambda, const float2 *P, const float2 *Q, const float2 *B,
                          const float2 *C, const float *log_dt, int H, int Nh, int L, float *K,
                          unsigned *flags, cudaStream_t st);

// ---- s4d.cu ----
cudaError_t launch_vandermonde(const float2 *A, const float2 *B, const float2 *C, const float *log_dt,
                               int H, int Nh, int L, float *K, unsigned *flags, cudaStream_t st);
cudaError_t launch_vandermonde_backward(const float2 *A, const float2 *B, const float2 *C, const float *log_dt,
                                        const float *dK, int H, int Nh, int L, float2 *dA, float2 *dB, float2 *dC,
                                        float *dlog_dt, cudaStream_t st);
cudaError_t launch_s4d_zoh(const float2 *A, const float2 *B, const float *log_dt, int H, int Nh,
                           float2 *Abar, float2 *Bbar, cudaStream_t st);

// ---- block.cu: the S4Block around the layer (norm, GLU projection, residual) ----
size_t glu_workspace_bytes(int H);
cudaError_t launch_layernorm_channels(const float *x, const float *gamma, const float *beta, float eps, int Bt,
                                      int H, int L, float *z, cudaStream_t st);
cudaError_t launch_glu_prepare(const float *W, int H, void *ws, cudaStream_t st);
cudaError_t launch_glu_projection(const float *y, const float *x, const float *bias, const void *ws, int Bt, int H,
                                  int L, float *out, unsigned *flags, cudaStream_t st);

// ---- zoh_dplr.cu: zero-order hold of the full DPLR system (Nh <= 32) ----
// K == nullptr: write Abar [H, N, N], Bbar [H, N], Cfull [H, N]; else the
// truncated kernel K [H, L]
cudaError_t launch_dplr_zoh(const float2 *Lambda, const float2 *P, const float2 *Q, const float2 *B,
                            const float2 *C, const float *log_dt, int H, int Nh, int L, float2 *Abar,
                            float2 *Bbar, float2 *Cfull, float *K, unsigned *flags, cudaStream_t st);

// ---- norm.cu: layer norm over token rows, and the backward over channels ----
size_t norm_backward_workspace_bytes(int D);
cudaError_t launch_layernorm_rows(int dtype, const void *x, const float *gamma, const float *beta, float eps,
                                  long long rows, int D, void *z, float *mean, float *rstd, cudaStream_t st);
cudaError_t launch_layernorm_rows_backward(int dtype, const void *dz, const void *x, const float *gamma,
                                           const float *mean, const float *rstd, long long rows, int D, void *dx,
                                           float *dgamma, float *dbeta, void *ws, cudaStream_t st);
cudaError_t launch_layernorm_channels_backward(const float *dz, const float *x, const float *gamma, float eps,
                                               int Bt, int H, int L, float *dx, float *dgamma, float *dbeta,
                                               void *ws, cudaStream_t st);

// ---- delta_scan.cu, delta_chunk.cu, delta_grad.cu: the gated delta rule ----
// n sequences; q, k, v with token strides sq, sk, sv (elements), o contiguous
struct DeltaArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    void *o;
    int n, hk, hv, dk, dv;
    long long sq, sk, sv;
    float scale;
    // the chunked form: n sequences of t tokens each, or between the offsets cu [n + 1]; tokens in all
    const int *cu;
    int t;
    long long tokens;
    int seg;   // chunks of a segment of a sequence; 0: sequences are not split
};
// T tokens for each sequence, state [n, hv, dk, dv] in place
cudaError_t launch_delta_scan(int dtype, const DeltaArgs &a, float *state, int T, cudaStream_t st);

// bytes of the images and factors of all chunks
size_t delta_prep_bytes(int dtype, long long tokens, int n, int hk, int hv, int dk);
// the chunks' images of T and PT and the gates' factors
cudaError_t launch_delta_prep(int dtype, const DeltaArgs &a, void *ws, unsigned *flags, cudaStream_t st);
// o and the last states; keep_s, keep_e (or null): the state before every chunk and E of every chunk.
// a.seg > 0: each sequence in segments, summaries: delta_segment_bytes of scratch
cudaError_t launch_delta_forward(int dtype, const DeltaArgs &a, const float *init, float *last, const void *ws,
                                 float *keep_s, float *keep_e, void *summaries, unsigned *flags, cudaStream_t st);
// whether splitting pays: chunks of a segment, or 0; *count: segments to keep room for, never fewer for more tokens
int delta_segment(long long tokens, int n, int hv, bool packed, long long *count);
size_t delta_segment_bytes(long long count, int hv, int dk, int dv, bool keep);
// the states before the segments from init; back: the states' gradients behind them from init
cudaError_t launch_delta_join(const DeltaArgs &a, const float *init, float *sums, bool keep, bool back, unsigned *flags,
                              cudaStream_t st);

// backward in the states: dV, the first states' gradient, keep_ds and keep_dr (behind every chunk, of every chunk)
cudaError_t launch_delta_backward(int dtype, const DeltaArgs &a, const void *dout, const float *dlast, float *dinit,
                                  const void *ws, void *dv, float *keep_ds, float *keep_dr, void *summaries,
                                  unsigned *flags, cudaStream_t st);
// the other gradients, from all that was kept
cudaError_t launch_delta_gradient(int dtype, const DeltaArgs &a, const void *dout, const void *ws, const float *keep_s,
                                  const float *keep_e, const float *keep_ds, const float *keep_dr, void *dq, void *dk,
                                  float *dg, float *dbeta, unsigned *flags, cudaStream_t st);

// ---- decode.cu ----
cudaError_t launch_dplr_discretize(const float2 *Lambda, const float2 *P, const float2 *Q,
                                   const float2 *B, const float2 *C, const float *log_dt, int H, int Nh,
                                   float2 *Abar, float2 *Bbar, float2 *Cfull, cudaStream_t st);
cudaError_t launch_dplr_discretize_structured(const float2 *Lambda, const float2 *P, const float2 *Q,
                                              const float2 *B, const float *log_dt, int H, int Nh,
                                              float2 *Astr, float2 *Bbar, cudaStream_t st);
cudaError_t launch_dplr_ctilde(const float2 *Lambda, const float2 *P, const float2 *Q, const float2 *C,
                               const float *log_dt, int H, int Nh, int L, float2 *Ct, cudaStream_t st);
cudaError_t launch_step(int mode, const float2 *Abar, const float2 *Bbar, const float2 *C, const float *D,
                        int Bt, int H, int Ns, int T, float2 *x, const float *u, float *y, cudaStream_t st);

}  // namespace s4
