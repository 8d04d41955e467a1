// block_api.cu -- the C ABI of the gated linear recurrence and of the norms around a mixer
// (include/ssd.h): host-side validation and dispatch, as in ssd_api.cu.  Every entry point
// validates all arguments before it enqueues anything and without a CUDA call.
#include <math.h>

#include "api_internal.h"
#include "kernels.h"

namespace {

using ssd::aligned;
using ssd::check_ptr;
using ssd::cuda_status;
using ssd::GlrDims;
using ssd::NormDims;
using bf16 = __nv_bfloat16;

constexpr int64_t kLim = (int64_t)1 << 30;  // any one extent
constexpr double kElems = 4e12;             // any one array, padding included
constexpr double kGrid = 2147483647.0;      // CTAs of a launch

bool known(ssd_dtype t) { return t == SSD_F32 || t == SSD_BF16; }
size_t size_of(ssd_dtype t) { return t == SSD_F32 ? 4 : 2; }

ssd_status check_glr(const ssd_glr_dims *dims, ssd_dtype dtype, bool step, bool grad, GlrDims *d) {
  if (!dims || !known(dtype)) return SSD_ERR_INVALID_ARG;
  const int64_t L = step ? 1 : dims->seqlen;
  if (dims->batch < 0 || dims->batch > kLim || L < 0 || L > kLim || dims->dim < 1 || dims->dim > kLim)
    return SSD_ERR_INVALID_ARG;
  const int64_t grad_stride = grad ? dims->grad_stride : dims->dim;
  if (dims->row_stride < dims->dim || grad_stride < dims->dim) return SSD_ERR_INVALID_ARG;
  const double tokens = (double)dims->batch * (double)L;
  if (tokens * (double)dims->row_stride > kElems || tokens * (double)grad_stride > kElems ||
      (double)dims->batch * (double)((dims->dim + 63) / 64) * 8 > kGrid)
    return SSD_ERR_INVALID_ARG;
  *d = GlrDims{dims->batch, L, dims->dim, dims->row_stride, grad_stride};
  return SSD_OK;
}

bool optional_ptr(const void *p, size_t align) { return p == nullptr || aligned(p, align); }

ssd_status check_norm(const ssd_norm_dims *dims, ssd_dtype dtype, ssd_dtype wide, float eps, bool gated, bool grad,
                      NormDims *d) {
  if (!dims || !known(dtype) || !known(wide)) return SSD_ERR_INVALID_ARG;
  if (dims->rows < 0 || dims->dim < 1 || dims->dim > kLim) return SSD_ERR_INVALID_ARG;
  const int64_t G = gated ? dims->ngroups : 1;
  if (G < 1 || dims->dim % G != 0 || (double)dims->rows * (double)G > kGrid) return SSD_ERR_INVALID_ARG;
  const int64_t gate = gated ? dims->gate_stride : dims->dim, dgate = gated && grad ? dims->dgate_stride : dims->dim;
  if (gate < dims->dim || dgate < dims->dim) return SSD_ERR_INVALID_ARG;
  if ((double)dims->rows * (double)gate > kElems || (double)dims->rows * (double)dgate > kElems)
    return SSD_ERR_INVALID_ARG;
  if (!(eps > 0.f) || !isfinite(eps)) return SSD_ERR_INVALID_ARG;
  if (dtype == SSD_F32 && wide == SSD_BF16) return SSD_ERR_UNSUPPORTED;
  *d = NormDims{dims->rows, dims->dim, G, gate, dgate};
  return SSD_OK;
}

// Calls f(TX{}, TR{}) with the element types of the pair (check_norm has refused the rest).
template <typename F>
cudaError_t by_types(ssd_dtype dtype, ssd_dtype wide, F f) {
  if (dtype == SSD_F32) return f(float{}, float{});
  if (wide == SSD_F32) return f(bf16{}, float{});
  return f(bf16{}, bf16{});
}

}  // namespace

extern "C" {

ssd_status ssd_glr_prefill(const ssd_glr_dims *dims, ssd_dtype dtype, const void *x, const void *r, const void *i,
                           const float *A, const float *initial_state, void *h, float *final_state,
                           ssd_stream_t stream) {
  GlrDims d;
  ssd_status s = check_glr(dims, dtype, false, false, &d);
  if (s != SSD_OK) return s;
  const int64_t n = d.b * d.L;
  const size_t e = size_of(dtype);
  if (!check_ptr(x, n, e) || !check_ptr(r, n, e) || !check_ptr(i, n, e) || !check_ptr(A, n, 4) || !check_ptr(h, n, e) ||
      !check_ptr(final_state, d.b, 4) || !optional_ptr(initial_state, 4))
    return SSD_ERR_INVALID_ARG;
  if (d.b == 0) return SSD_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d.L == 0) {  // no tokens: the state carries over unchanged
    const size_t bytes = (size_t)d.b * d.D * sizeof(float);
    if (initial_state == final_state) return SSD_OK;
    if (initial_state == nullptr) return cuda_status(cudaMemsetAsync(final_state, 0, bytes, st));
    return cuda_status(cudaMemcpyAsync(final_state, initial_state, bytes, cudaMemcpyDeviceToDevice, st));
  }
  if (dtype == SSD_F32)
    return cuda_status(ssd::launch_glr_prefill<float>(
        static_cast<const float *>(x), static_cast<const float *>(r), static_cast<const float *>(i), A, initial_state,
        static_cast<float *>(h), final_state, d, st));
  return cuda_status(ssd::launch_glr_prefill<bf16>(static_cast<const bf16 *>(x), static_cast<const bf16 *>(r),
                                                   static_cast<const bf16 *>(i), A, initial_state,
                                                   static_cast<bf16 *>(h), final_state, d, st));
}

ssd_status ssd_glr_decode_step(const ssd_glr_dims *dims, ssd_dtype dtype, float *state, const void *x, const void *r,
                               const void *i, const float *A, void *h, ssd_stream_t stream) {
  GlrDims d;
  ssd_status s = check_glr(dims, dtype, true, false, &d);
  if (s != SSD_OK) return s;
  const size_t e = size_of(dtype);
  if (!check_ptr(state, d.b, 4) || !check_ptr(x, d.b, e) || !check_ptr(r, d.b, e) || !check_ptr(i, d.b, e) ||
      !check_ptr(A, d.b, 4) || !check_ptr(h, d.b, e))
    return SSD_ERR_INVALID_ARG;
  if (d.b == 0) return SSD_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == SSD_F32)
    return cuda_status(ssd::launch_glr_decode_step<float>(
        state, static_cast<const float *>(x), static_cast<const float *>(r), static_cast<const float *>(i), A,
        static_cast<float *>(h), d, st));
  return cuda_status(ssd::launch_glr_decode_step<bf16>(state, static_cast<const bf16 *>(x),
                                                       static_cast<const bf16 *>(r), static_cast<const bf16 *>(i), A,
                                                       static_cast<bf16 *>(h), d, st));
}

ssd_status ssd_glr_wait_selftest(float *out, size_t out_bytes, int ranks, int tiles, int late_rank, int late_tile,
                                 uint64_t delay_ns, uint64_t limit_ns, ssd_stream_t stream) {
  if (ranks < 2 || ranks > 8 || tiles < 1 || tiles > 64 || late_rank < -1 || late_rank >= ranks || late_tile < 0 ||
      late_tile >= tiles || delay_ns > 100000000ull || limit_ns == 0 || limit_ns > 100000000ull)
    return SSD_ERR_INVALID_ARG;
  if (!check_ptr(out, 1, 8) || out_bytes < (size_t)tiles * ranks * 4 * 64 * sizeof(float)) return SSD_ERR_INVALID_ARG;
  return cuda_status(ssd::launch_glr_wait_selftest(out, ranks, tiles, late_rank, late_tile, delay_ns, limit_ns,
                                                   reinterpret_cast<cudaStream_t>(stream)));
}

size_t ssd_glr_backward_workspace_size(const ssd_glr_dims *dims, ssd_dtype dtype) {
  GlrDims d;
  if (check_glr(dims, dtype, false, true, &d) != SSD_OK || d.b == 0 || d.L == 0) return 0;
  return ssd::glr_backward_floats(d) * sizeof(float);
}

ssd_status ssd_glr_backward(const ssd_glr_dims *dims, ssd_dtype dtype, const void *x, const void *r, const void *i,
                            const float *A, const float *initial_state, const void *h, const void *dh,
                            const float *dfinal_state, void *dx, void *dr, void *di, float *dA, float *dinitial_state,
                            void *workspace, size_t workspace_bytes, ssd_stream_t stream) {
  GlrDims d;
  ssd_status s = check_glr(dims, dtype, false, true, &d);
  if (s != SSD_OK) return s;
  const int64_t n = d.b * d.L;
  const size_t e = size_of(dtype);
  for (const void *p : {x, r, i, h, dh, (const void *)dx, (const void *)dr, (const void *)di})
    if (!check_ptr(p, n, e)) return SSD_ERR_INVALID_ARG;
  if (!check_ptr(A, n, 4) || !check_ptr(dA, d.D, 4) || !optional_ptr(initial_state, 4) ||
      !optional_ptr(dfinal_state, 4) || !optional_ptr(dinitial_state, 4))
    return SSD_ERR_INVALID_ARG;
  const size_t need = ssd_glr_backward_workspace_size(dims, dtype);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (n == 0) {  // no tokens: no sums, and the state's gradient passes through
    cudaError_t err = cudaMemsetAsync(dA, 0, (size_t)d.D * sizeof(float), st);
    const size_t bytes = (size_t)d.b * d.D * sizeof(float);
    if (err == cudaSuccess && bytes > 0 && dinitial_state != nullptr && dinitial_state != dfinal_state)
      err = dfinal_state == nullptr
                ? cudaMemsetAsync(dinitial_state, 0, bytes, st)
                : cudaMemcpyAsync(dinitial_state, dfinal_state, bytes, cudaMemcpyDeviceToDevice, st);
    return cuda_status(err);
  }
  float *part = static_cast<float *>(workspace);
  if (dtype == SSD_F32)
    return cuda_status(ssd::launch_glr_backward<float>(
        static_cast<const float *>(x), static_cast<const float *>(r), static_cast<const float *>(i), A, initial_state,
        static_cast<const float *>(h), static_cast<const float *>(dh), dfinal_state, static_cast<float *>(dx),
        static_cast<float *>(dr), static_cast<float *>(di), dA, dinitial_state, part, d, st));
  return cuda_status(ssd::launch_glr_backward<bf16>(
      static_cast<const bf16 *>(x), static_cast<const bf16 *>(r), static_cast<const bf16 *>(i), A, initial_state,
      static_cast<const bf16 *>(h), static_cast<const bf16 *>(dh), dfinal_state, static_cast<bf16 *>(dx),
      static_cast<bf16 *>(dr), static_cast<bf16 *>(di), dA, dinitial_state, part, d, st));
}

ssd_status ssd_residual_norm(const ssd_norm_dims *dims, ssd_dtype dtype, ssd_dtype residual_dtype, const void *x,
                             const float *scale, const void *residual, const float *weight, float eps,
                             void *residual_out, void *out, ssd_stream_t stream) {
  NormDims d;
  ssd_status s = check_norm(dims, dtype, residual_dtype, eps, false, false, &d);
  if (s != SSD_OK) return s;
  const size_t e = size_of(dtype), f = size_of(residual_dtype);
  if (!check_ptr(x, d.rows, e) || !check_ptr(out, d.rows, e) || !check_ptr(weight, d.rows, 4) ||
      !optional_ptr(scale, 4) || !optional_ptr(residual, f) || !optional_ptr(residual_out, f))
    return SSD_ERR_INVALID_ARG;
  if (d.rows == 0) return SSD_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(by_types(dtype, residual_dtype, [&](auto tx, auto tr) {
    using TX = decltype(tx);
    using TR = decltype(tr);
    return ssd::launch_residual_norm<TX, TR>(static_cast<const TX *>(x), scale, static_cast<const TR *>(residual),
                                             weight, eps, static_cast<TR *>(residual_out), static_cast<TX *>(out), d,
                                             st);
  }));
}

size_t ssd_norm_backward_workspace_size(const ssd_norm_dims *dims) {
  if (!dims || dims->rows <= 0 || (double)dims->rows > kGrid || dims->dim < 1 || dims->dim > kLim) return 0;
  return ssd::norm_backward_floats(NormDims{dims->rows, dims->dim, 1, dims->dim, dims->dim}) * sizeof(float);
}

ssd_status ssd_residual_norm_backward(const ssd_norm_dims *dims, ssd_dtype dtype, ssd_dtype residual_dtype,
                                      const void *x, const float *scale, const void *s_in, const float *weight,
                                      float eps, const void *dout, const void *dresidual_out, void *dx,
                                      void *dresidual, float *dweight, float *dscale, void *workspace,
                                      size_t workspace_bytes, ssd_stream_t stream) {
  NormDims d;
  ssd_status s = check_norm(dims, dtype, residual_dtype, eps, false, true, &d);
  if (s != SSD_OK) return s;
  const size_t e = size_of(dtype), f = size_of(residual_dtype);
  if (!check_ptr(s_in, d.rows, f) || !check_ptr(dout, d.rows, e) || !check_ptr(weight, d.rows, 4) ||
      !check_ptr(x, dscale != nullptr ? d.rows : 0, e) || !optional_ptr(x, e) || !optional_ptr(scale, 4) ||
      !optional_ptr(dresidual_out, f) || !optional_ptr(dx, e) || !optional_ptr(dresidual, f) ||
      !optional_ptr(dweight, 4) || !optional_ptr(dscale, 4))
    return SSD_ERR_INVALID_ARG;
  const size_t need = ssd_norm_backward_workspace_size(dims);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d.rows == 0) {  // no rows: empty sums
    cudaError_t err = cudaSuccess;
    for (float *p : {dweight, dscale})
      if (err == cudaSuccess && p != nullptr) err = cudaMemsetAsync(p, 0, (size_t)d.D * sizeof(float), st);
    return cuda_status(err);
  }
  return cuda_status(by_types(dtype, residual_dtype, [&](auto tx, auto tr) {
    using TX = decltype(tx);
    using TR = decltype(tr);
    return ssd::launch_residual_norm_backward<TX, TR>(
        static_cast<const TX *>(x), scale, static_cast<const TR *>(s_in), weight, eps, static_cast<const TX *>(dout),
        static_cast<const TR *>(dresidual_out), static_cast<TX *>(dx), static_cast<TR *>(dresidual), dweight, dscale,
        static_cast<float *>(workspace), d, st);
  }));
}

ssd_status ssd_gated_norm(const ssd_norm_dims *dims, ssd_dtype dtype, ssd_dtype y_dtype, int gate_first, const void *y,
                          const void *z, const float *weight, float eps, void *out, ssd_stream_t stream) {
  NormDims d;
  ssd_status s = check_norm(dims, dtype, y_dtype, eps, true, false, &d);
  if (s != SSD_OK) return s;
  const size_t e = size_of(dtype), f = size_of(y_dtype);
  if (!check_ptr(y, d.rows, f) || !check_ptr(z, d.rows, e) || !check_ptr(weight, d.rows, 4) ||
      !check_ptr(out, d.rows, e))
    return SSD_ERR_INVALID_ARG;
  if (d.rows == 0) return SSD_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return cuda_status(by_types(dtype, y_dtype, [&](auto tx, auto tr) {
    using TX = decltype(tx);
    using TR = decltype(tr);
    return ssd::launch_gated_norm<TX, TR>(gate_first != 0, static_cast<const TR *>(y), static_cast<const TX *>(z),
                                          weight, eps, static_cast<TX *>(out), d, st);
  }));
}

ssd_status ssd_gated_norm_backward(const ssd_norm_dims *dims, ssd_dtype dtype, ssd_dtype y_dtype, int gate_first,
                                   const void *y, const void *z, const float *weight, float eps, const void *dout,
                                   void *dy, void *dz, float *dweight, void *workspace, size_t workspace_bytes,
                                   ssd_stream_t stream) {
  NormDims d;
  ssd_status s = check_norm(dims, dtype, y_dtype, eps, true, true, &d);
  if (s != SSD_OK) return s;
  const size_t e = size_of(dtype), f = size_of(y_dtype);
  if (!check_ptr(y, d.rows, f) || !check_ptr(z, d.rows, e) || !check_ptr(weight, d.rows, 4) ||
      !check_ptr(dout, d.rows, e) || !optional_ptr(dy, f) || !optional_ptr(dz, e) || !optional_ptr(dweight, 4))
    return SSD_ERR_INVALID_ARG;
  const size_t need = ssd_norm_backward_workspace_size(dims);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d.rows == 0)
    return dweight == nullptr ? SSD_OK : cuda_status(cudaMemsetAsync(dweight, 0, (size_t)d.D * sizeof(float), st));
  return cuda_status(by_types(dtype, y_dtype, [&](auto tx, auto tr) {
    using TX = decltype(tx);
    using TR = decltype(tr);
    return ssd::launch_gated_norm_backward<TX, TR>(
        gate_first != 0, static_cast<const TR *>(y), static_cast<const TX *>(z), weight, eps,
        static_cast<const TX *>(dout), static_cast<TR *>(dy), static_cast<TX *>(dz), dweight,
        static_cast<float *>(workspace), d, st);
  }));
}

}  // extern "C"
