// kernels.h -- host-side launchers of the libssd kernels (internal to the library).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include "common.cuh"

namespace ssd {

// Launches f; the status is this launch's own.
template <typename... P, typename... V>
cudaError_t launch(void (*f)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, bool dependent, V... v) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, f, P(v)...);
}

// The same as a programmatic dependent of what the stream ran before: its CTAs take their places as the last ones of
// that kernel leave theirs, and f itself waits (grid_dep_wait, before it touches memory) until that kernel is complete.
// f's pointers are not __restrict__: what they point to may change until that wait, and the qualifier would let the
// compiler load it before, or as data that is read-only for all of the kernel.
template <typename... P, typename... V>
cudaError_t launch_dependent(void (*f)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, V... v) {
  return launch(f, grid, threads, smem, st, true, v...);
}

// prefill_simt.cu
cudaError_t launch_dA_cumsum(const float *dt, const float *A, float *cum, const Dims &d, int Q, int nc,
                             cudaStream_t st);
template <typename T>
cudaError_t launch_chunk_state_simt(const T *x, const float *dt, const T *B, const float *cum, float *states,
                                    const Dims &d, int Q, int nc, cudaStream_t st);
// init: state before the first token (NULL: zero); cstates: state after each chunk (NULL: not written)
cudaError_t launch_state_passing(float *states, const float *cum, const float *init, float *final_state,
                                 float *cstates, const Dims &d, int Q, int nc, cudaStream_t st);
template <typename T>
cudaError_t launch_chunk_scan_simt(const T *x, const float *dt, const T *B, const T *C, const float *D,
                                   const float *cum, const float *hprev, float *y, const Dims &d, int Q, int nc,
                                   cudaStream_t st);
size_t chunk_scan_simt_smem_bytes(int N);

// prefill_tc.cu (bf16 x/B/C, P = 64, N = 128, Q in {128, 256})
bool tc_prefill_supported(const Dims &d, int Q);
// floats of the per-(batch, head, chunk) decay table the tensor-core kernels share
size_t tc_prefill_table_floats(const Dims &d, int Q, int nc);
cudaError_t launch_tc_prefill(const __nv_bfloat16 *x, const float *dt, const float *A, const __nv_bfloat16 *B,
                              const __nv_bfloat16 *C, const float *D, const float *init, float *y, float *final_state,
                              float *cstates, float *tab, float *states, float *cdecay, __nv_bfloat16 *hprev, int *err,
                              const Dims &d, int Q, int nc, cudaStream_t st, const cudaEvent_t *ev);

// decode.cu
template <typename T>
cudaError_t launch_decode_step(float *state, const T *x, const float *dt, const float *A, const T *B,
                               const T *C, const float *D, float *y, const Dims &d, cudaStream_t st);

// frontend.cu: conv + SiLU + split, softplus dt; the new conv state when state_out != NULL
template <typename T>
cudaError_t launch_frontend(const T *xbc, const float *w, const float *bias, const float *state_in,
                            float *state_out, const float *dt_raw, const float *dt_bias, T *x, T *B, T *C, float *dt,
                            const Dims &d, cudaStream_t st);

// decode_window.cu (window length 1 .. 16)
template <typename T>
cudaError_t launch_decode_window_step(const float *state, T *win_x, float *win_dt, T *win_B, int W, int pos,
                                      const T *x, const float *dt, const float *A, const T *B, const T *C,
                                      const float *D, float *y, const Dims &d, cudaStream_t st);
template <typename T>
cudaError_t launch_decode_window_flush(float *state, const T *win_x, const float *win_dt, const T *win_B, int W,
                                       int count, const float *A, const Dims &d, cudaStream_t st);

// Sizes of a gated linear recurrence (glr.cu): strides in elements.
struct GlrDims {
  int64_t b, L, D;
  int64_t row;   // between consecutive tokens of x, r, i
  int64_t grad;  // between consecutive tokens of dx, dr, di
};

// glr.cu
template <typename T>
cudaError_t launch_glr_prefill(const T *x, const T *r, const T *i, const float *A, const float *init, T *h,
                               float *final_state, const GlrDims &d, cudaStream_t st);
template <typename T>
cudaError_t launch_glr_decode_step(float *state, const T *x, const T *r, const T *i, const float *A, T *h,
                                   const GlrDims &d, cudaStream_t st);
cudaError_t launch_glr_wait_selftest(float *out, int ranks, int tiles, int late_rank, int late_tile, uint64_t delay,
                                     uint64_t limit, cudaStream_t st);
// floats of scratch: the partial sums of dA
size_t glr_backward_floats(const GlrDims &d);
template <typename T>
cudaError_t launch_glr_backward(const T *x, const T *r, const T *i, const float *A, const float *init, const T *h,
                                const T *dh, const float *dfinal, T *dx, T *dr, T *di, float *dA, float *dinit,
                                float *part, const GlrDims &d, cudaStream_t st);

// Sizes of the norms (norm.cu); the residual norm has one group.
struct NormDims {
  int64_t rows, D, G;
  int64_t gate, dgate;  // elements between rows of z and of dz
};

// norm.cu.  TX: x, z, out, dout; TR: residual stream or y.
template <typename TX, typename TR>
cudaError_t launch_residual_norm(const TX *x, const float *scale, const TR *res, const float *w, float eps,
                                 TR *res_out, TX *out, const NormDims &d, cudaStream_t st);
// One or two (o1 != NULL) vectors of D as the sums of n rows each, in a fixed order; a programmatic dependent of the
// kernel that writes the rows.
cudaError_t launch_row_sums(const float *p0, const float *p1, float *o0, float *o1, int64_t D, int64_t n,
                            cudaStream_t st);
// floats of scratch: the partial sums of two vectors of dim
size_t norm_backward_floats(const NormDims &d);
template <typename TX, typename TR>
cudaError_t launch_residual_norm_backward(const TX *x, const float *scale, const TR *s, const float *w, float eps,
                                          const TX *dout, const TR *dres_out, TX *dx, TR *dres, float *dw,
                                          float *dscale, float *part, const NormDims &d, cudaStream_t st);
template <typename TX, typename TR>
cudaError_t launch_gated_norm(bool gate_first, const TR *y, const TX *z, const float *w, float eps, TX *out,
                              const NormDims &d, cudaStream_t st);
template <typename TX, typename TR>
cudaError_t launch_gated_norm_backward(bool gate_first, const TR *y, const TX *z, const float *w, float eps,
                                       const TX *dout, TR *dy, TX *dz, float *dw, float *part, const NormDims &d,
                                       cudaStream_t st);

}  // namespace ssd
