// norm.cu -- the norms around a mixer and their gradients: the residual norm before it (residual add, scale of the
// branch, RMS norm) and the gated norm after it (silu gate, RMS norm over each group of channels).  Statistics and
// sums over rows are fp32.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace ssd {

namespace {

constexpr int kThreads = 256;
constexpr int kParts = 296;  // most rows of partial sums: two CTAs for each SM

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// The sum over a CTA, in every thread.
__device__ __forceinline__ float block_sum(float v, float *sh) {
  v = warp_sum(v, 32);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int k = 0; k < kThreads / 32; ++k) v += sh[k];
  return v;
}

enum Mode { kResidual, kGateFirst, kNormFirst };

// One CTA per (row, group): a pass for the mean square, one that writes.
template <Mode M, typename TX, typename TR>
__global__ void __launch_bounds__(kThreads)
    k_norm(const TX *x, const float *__restrict__ scale, const TR *wide, const float *__restrict__ w, float eps,
           TR *wide_out, TX *out, NormDims d) {
  __shared__ float sh[kThreads / 32];
  const int64_t row = blockIdx.x / d.G, W = d.D / d.G, c0 = (blockIdx.x % d.G) * W;
  const TX *xr = x + row * (M == kResidual ? d.D : d.gate);
  auto value = [&](int64_t c) {
    if (M == kResidual) {
      const float v = scale != nullptr ? scale[c] * to_f32(xr[c]) : to_f32(xr[c]);
      return wide != nullptr ? v + to_f32(wide[row * d.D + c]) : v;
    }
    const float y = to_f32(wide[row * d.D + c]);
    if (M == kNormFirst) return y;
    const float z = to_f32(xr[c]);
    return y * z * sigmoid(z);
  };
  float ss = 0.f;
  for (int64_t c = c0 + threadIdx.x; c < c0 + W; c += kThreads) {
    const float v = value(c);
    ss = fmaf(v, v, ss);
  }
  const float rstd = rsqrtf(block_sum(ss, sh) / (float)W + eps);
  for (int64_t c = c0 + threadIdx.x; c < c0 + W; c += kThreads) {
    const float v = value(c);
    float o = v * rstd * w[c];
    if (M == kNormFirst) {
      const float z = to_f32(xr[c]);
      o *= z * sigmoid(z);
    }
    if (M == kResidual && wide_out != nullptr) wide_out[row * d.D + c] = from_f32<TR>(v);
    out[row * d.D + c] = from_f32<TX>(o);
  }
}

// Gradients.  A CTA takes rows blockIdx.x, + gridDim.x, ...; a column belongs to one thread of it, which adds the
// row's terms to the CTA's partial sums.
//   kResidual: wide = s, dwide = dresidual_out, x for dscale; writes dx, dwide_out = dresidual
//   gated:     wide = y, x = z;                                writes dx = dz, dwide_out = dy
template <Mode M, typename TX, typename TR>
__global__ void __launch_bounds__(kThreads)
    k_norm_backward(const TX *__restrict__ x, const float *__restrict__ scale, const TR *__restrict__ wide,
                    const float *__restrict__ w, float eps, const TX *__restrict__ dout, const TR *dwide, TX *dx,
                    TR *dwide_out, float *__restrict__ pw, float *__restrict__ ps, NormDims d) {
  __shared__ float sh[kThreads / 32];
  const int64_t W = d.D / d.G;
  float *pwr = pw != nullptr ? pw + blockIdx.x * d.D : nullptr, *psr = ps != nullptr ? ps + blockIdx.x * d.D : nullptr;
  for (int64_t c = threadIdx.x; c < W; c += kThreads)
    for (int64_t g = 0; g < d.G; ++g) {
      if (pwr != nullptr) pwr[g * W + c] = 0.f;
      if (psr != nullptr) psr[g * W + c] = 0.f;
    }
  for (int64_t row = blockIdx.x; row < d.rows; row += gridDim.x)
    for (int64_t c0 = 0; c0 < d.D; c0 += W) {
      const TX *xr = x + row * (M == kResidual ? d.D : d.gate);
      const TR *yr = wide + row * d.D;
      const TX *ur = dout + row * d.D;
      // v: what is normed; un: the gradient of the weighted norm
      auto load = [&](int64_t c, float &v, float &un, float &y, float &z, float &sg) {
        y = to_f32(yr[c]);
        un = to_f32(ur[c]);
        v = y;
        z = sg = 0.f;
        if (M != kResidual) {
          z = to_f32(xr[c]);
          sg = sigmoid(z);
          if (M == kGateFirst) v = y * z * sg;
          if (M == kNormFirst) un *= z * sg;
        }
      };
      float ss = 0.f, dot = 0.f, v, un, y, z, sg;
      for (int64_t c = c0 + threadIdx.x; c < c0 + W; c += kThreads) {
        load(c, v, un, y, z, sg);
        ss = fmaf(v, v, ss);
        dot = fmaf(un * w[c], v, dot);
      }
      const float rstd = rsqrtf(block_sum(ss, sh) / (float)W + eps);
      const float mean = block_sum(dot, sh) * rstd / (float)W;  // of (w dout) n
      for (int64_t c = c0 + threadIdx.x; c < c0 + W; c += kThreads) {
        load(c, v, un, y, z, sg);
        const float n = v * rstd;
        float dv = rstd * (un * w[c] - n * mean);
        if (M == kResidual) {
          if (dwide != nullptr) dv += to_f32(dwide[row * d.D + c]);
          if (psr != nullptr) psr[c] += dv * to_f32(xr[c]);
          if (dx != nullptr) dx[row * d.D + c] = from_f32<TX>(scale != nullptr ? dv * scale[c] : dv);
          if (dwide_out != nullptr) dwide_out[row * d.D + c] = from_f32<TR>(dv);
        } else {
          const float slope = sg * (1.f + z * (1.f - sg));
          if (dx != nullptr)
            dx[row * d.dgate + c] = from_f32<TX>((M == kGateFirst ? dv * y : to_f32(ur[c]) * n * w[c]) * slope);
          if (dwide_out != nullptr) dwide_out[row * d.D + c] = from_f32<TR>(M == kGateFirst ? dv * z * sg : dv);
        }
        if (pwr != nullptr) pwr[c] += un * n;
      }
    }
}

// The partial sums of one or two vectors, in order.
__global__ void __launch_bounds__(128) k_norm_sum(const float *__restrict__ pw, const float *__restrict__ ps, float *dw,
                                                  float *ds, int64_t D, int n) {
  const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x;
  const float *p = blockIdx.y == 0 ? pw : ps;
  float *o = blockIdx.y == 0 ? dw : ds;
  if (c >= D || o == nullptr) return;
  float s = 0.f;
  for (int k = 0; k < n; ++k) s += p[k * D + c];
  o[c] = s;
}

int parts_of(const NormDims &d) { return (int)std::min<int64_t>(d.rows, kParts); }

template <Mode M, typename TX, typename TR>
cudaError_t norm(const TX *x, const float *scale, const TR *wide, const float *w, float eps, TR *wide_out, TX *out,
                 const NormDims &d, cudaStream_t st) {
  k_norm<M, TX, TR><<<(unsigned)(d.rows * d.G), kThreads, 0, st>>>(x, scale, wide, w, eps, wide_out, out, d);
  return cudaGetLastError();
}

template <Mode M, typename TX, typename TR>
cudaError_t norm_backward(const TX *x, const float *scale, const TR *wide, const float *w, float eps, const TX *dout,
                          const TR *dwide, TX *dx, TR *dwide_out, float *dw, float *ds, float *part, const NormDims &d,
                          cudaStream_t st) {
  const int parts = parts_of(d);
  float *pw = dw != nullptr ? part : nullptr, *ps = ds != nullptr ? part + (int64_t)parts * d.D : nullptr;
  k_norm_backward<M, TX, TR><<<parts, kThreads, 0, st>>>(x, scale, wide, w, eps, dout, dwide, dx, dwide_out, pw, ps, d);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (dw == nullptr && ds == nullptr)) return e;
  k_norm_sum<<<dim3((unsigned)((d.D + 127) / 128), 2), 128, 0, st>>>(pw, ps, dw, ds, d.D, parts);
  return cudaGetLastError();
}

}  // namespace

size_t norm_backward_floats(const NormDims &d) { return (size_t)2 * parts_of(d) * d.D; }

template <typename TX, typename TR>
cudaError_t launch_residual_norm(const TX *x, const float *scale, const TR *res, const float *w, float eps,
                                 TR *res_out, TX *out, const NormDims &d, cudaStream_t st) {
  return norm<kResidual, TX, TR>(x, scale, res, w, eps, res_out, out, d, st);
}

template <typename TX, typename TR>
cudaError_t launch_residual_norm_backward(const TX *x, const float *scale, const TR *s, const float *w, float eps,
                                          const TX *dout, const TR *dres_out, TX *dx, TR *dres, float *dw,
                                          float *dscale, float *part, const NormDims &d, cudaStream_t st) {
  return norm_backward<kResidual, TX, TR>(x, scale, s, w, eps, dout, dres_out, dx, dres, dw, dscale, part, d, st);
}

template <typename TX, typename TR>
cudaError_t launch_gated_norm(bool gate_first, const TR *y, const TX *z, const float *w, float eps, TX *out,
                              const NormDims &d, cudaStream_t st) {
  return gate_first ? norm<kGateFirst, TX, TR>(z, nullptr, y, w, eps, nullptr, out, d, st)
                    : norm<kNormFirst, TX, TR>(z, nullptr, y, w, eps, nullptr, out, d, st);
}

template <typename TX, typename TR>
cudaError_t launch_gated_norm_backward(bool gate_first, const TR *y, const TX *z, const float *w, float eps,
                                       const TX *dout, TR *dy, TX *dz, float *dw, float *part, const NormDims &d,
                                       cudaStream_t st) {
  const TR *none = nullptr;
  return gate_first
             ? norm_backward<kGateFirst, TX, TR>(z, nullptr, y, w, eps, dout, none, dz, dy, dw, nullptr, part, d, st)
             : norm_backward<kNormFirst, TX, TR>(z, nullptr, y, w, eps, dout, none, dz, dy, dw, nullptr, part, d, st);
}

#define SSD_NORM_INSTANCES(TX, TR)                                                                                    \
  template cudaError_t launch_residual_norm<TX, TR>(const TX *, const float *, const TR *, const float *, float, TR *, \
                                                    TX *, const NormDims &, cudaStream_t);                            \
  template cudaError_t launch_residual_norm_backward<TX, TR>(                                                         \
      const TX *, const float *, const TR *, const float *, float, const TX *, const TR *, TX *, TR *, float *,       \
      float *, float *, const NormDims &, cudaStream_t);                                                              \
  template cudaError_t launch_gated_norm<TX, TR>(bool, const TR *, const TX *, const float *, float, TX *,            \
                                                 const NormDims &, cudaStream_t);                                     \
  template cudaError_t launch_gated_norm_backward<TX, TR>(bool, const TR *, const TX *, const float *, float,         \
                                                          const TX *, TR *, TX *, float *, float *, const NormDims &, \
                                                          cudaStream_t);
SSD_NORM_INSTANCES(float, float)
SSD_NORM_INSTANCES(__nv_bfloat16, float)
SSD_NORM_INSTANCES(__nv_bfloat16, __nv_bfloat16)

}  // namespace ssd
