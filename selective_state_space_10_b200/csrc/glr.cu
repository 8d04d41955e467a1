// glr.cu -- the gated linear recurrence, one state value per channel:
//
//   L_t = A sigmoid(r_t),  a_t = exp(L_t),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t
//
// over whole sequences, for one token, and its gradients.
#include "common.cuh"
#include "kernels.h"

namespace ssd {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float sqrt_approx(float v) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rsqrt_approx(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// a = exp(L) and 1 - a^2 for L <= 0.  Near zero u = exp(L) - 1 comes from its Taylor series
// (the first term left out is below 0.5^8 / 9! = 1e-8 of the sum), so that a = 1 + u and
// 1 - a^2 = -u (2 + u) keep full relative precision for decays close to 1; an exp(L) rounded
// near 1 and subtracted would not, and its error would be carried through every step of a
// long memory.  Further away the exponential itself keeps a small a precise.
__device__ __forceinline__ void decay(float L, float &a, float &rest) {
  float p = 1.f / 40320.f;
  p = fmaf(p, L, 1.f / 5040.f);
  p = fmaf(p, L, 1.f / 720.f);
  p = fmaf(p, L, 1.f / 120.f);
  p = fmaf(p, L, 1.f / 24.f);
  p = fmaf(p, L, 1.f / 6.f);
  p = fmaf(p, L, 0.5f);
  p = fmaf(p, L, 1.f);
  p *= L;
  const bool far = L < -0.5f;
  const float e = ex2(L * kLog2e), u = far ? e - 1.f : p;
  a = far ? e : 1.f + p;
  rest = -u * (2.f + u);
}

// The smaller of sigmoid(v) and sigmoid(-v); the other is one minus it.  exp(-|v|) cannot
// overflow, and neither side loses relative precision.
__device__ __forceinline__ float sigmoid_small(float v) {
  const float e = ex2(-fabsf(v) * kLog2e);
  return e * rcp(1.f + e);
}
__device__ __forceinline__ float pick(float v, float small) { return v >= 0.f ? 1.f - small : small; }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// One step: the decay a and the input term b = sqrt(1 - a^2) sigmoid(i) x.
__device__ __forceinline__ void gate(float x, float r, float i, float A, float &a, float &b) {
  float rest;
  decay(A * pick(r, sigmoid_small(r)), a, rest);
  b = sqrt_approx(rest) * pick(i, sigmoid_small(i)) * x;
}

// One thread per (batch row, channel), walking the sequence.
template <typename T>
__global__ void __launch_bounds__(128) k_glr_prefill(const T *__restrict__ x, const T *__restrict__ r,
                                                     const T *__restrict__ i, const float *__restrict__ A,
                                                     const float *init, T *__restrict__ h, float *final_state,
                                                     GlrDims d, int blocks) {
  const int64_t b = blockIdx.x / blocks, c = (int64_t)(blockIdx.x % blocks) * 128 + threadIdx.x;
  if (c >= d.D) return;
  const float Ac = A[c];
  float s = init != nullptr ? init[b * d.D + c] : 0.f;
  for (int64_t t = 0; t < d.L; ++t) {
    const int64_t at = (b * d.L + t) * d.row + c;
    float a, v;
    gate(to_f32(x[at]), to_f32(r[at]), to_f32(i[at]), Ac, a, v);
    s = fmaf(a, s, v);
    h[(b * d.L + t) * d.D + c] = from_f32<T>(s);
  }
  final_state[b * d.D + c] = s;
}

template <typename T>
__global__ void __launch_bounds__(128) k_glr_decode(float *__restrict__ state, const T *__restrict__ x,
                                                    const T *__restrict__ r, const T *__restrict__ i,
                                                    const float *__restrict__ A, T *__restrict__ h, GlrDims d,
                                                    int blocks) {
  const int64_t b = blockIdx.x / blocks, c = (int64_t)(blockIdx.x % blocks) * 128 + threadIdx.x;
  if (c >= d.D) return;
  const int64_t at = b * d.row + c, s = b * d.D + c;
  float a, v;
  gate(to_f32(x[at]), to_f32(r[at]), to_f32(i[at]), A[c], a, v);
  const float n = fmaf(a, state[s], v);
  state[s] = n;
  h[s] = from_f32<T>(n);
}

// The reverse walk: c_t = a_t g_t with g_t = dh_t + c_{t+1}.
template <typename T>
__global__ void __launch_bounds__(128)
    k_glr_backward(const T *__restrict__ x, const T *__restrict__ r, const T *__restrict__ i,
                   const float *__restrict__ A, const float *__restrict__ init, const T *__restrict__ h,
                   const T *__restrict__ dh, const float *dfinal, T *__restrict__ dx, T *__restrict__ dr,
                   T *__restrict__ di, float *dinit, float *__restrict__ part, GlrDims d, int blocks) {
  const int64_t b = blockIdx.x / blocks, c = (int64_t)(blockIdx.x % blocks) * 128 + threadIdx.x;
  if (c >= d.D) return;
  const float Ac = A[c];
  float carry = dfinal != nullptr ? dfinal[b * d.D + c] : 0.f, dA = 0.f;
  for (int64_t t = d.L - 1; t >= 0; --t) {
    const int64_t at = (b * d.L + t) * d.row + c, to = (b * d.L + t) * d.grad + c, o = (b * d.L + t) * d.D + c;
    const float xv = to_f32(x[at]), rv = to_f32(r[at]), iv = to_f32(i[at]);
    const float before = t > 0 ? to_f32(h[o - d.D]) : init != nullptr ? init[b * d.D + c] : 0.f;
    const float zr = sigmoid_small(rv), zi = sigmoid_small(iv), sr = pick(rv, zr), si = pick(iv, zi);
    const float Lt = Ac * sr;
    float a, b2;
    decay(Lt, a, b2);
    const float inv = b2 > 1e-37f ? rsqrt_approx(b2) : 0.f, beta = b2 * inv;
    const float g = to_f32(dh[o]) + carry;
    const float gx = g * beta * si;
    const float dL = g * (a * before - a * a * inv * si * xv);
    dx[to] = from_f32<T>(gx);
    di[to] = from_f32<T>(gx * xv * pick(-iv, zi));
    dr[to] = from_f32<T>(dL * Lt * pick(-rv, zr));
    dA = fmaf(dL, sr, dA);
    carry = a * g;
  }
  part[b * d.D + c] = dA;
  if (dinit != nullptr) dinit[b * d.D + c] = carry;
}

// dA over the batch, in order.
__global__ void __launch_bounds__(128) k_glr_sum(const float *__restrict__ part, float *__restrict__ dA, int64_t D,
                                                 int64_t n) {
  const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (c >= D) return;
  float s = 0.f;
  for (int64_t k = 0; k < n; ++k) s += part[k * D + c];
  dA[c] = s;
}

}  // namespace

template <typename T>
cudaError_t launch_glr_prefill(const T *x, const T *r, const T *i, const float *A, const float *init, T *h,
                               float *final_state, const GlrDims &d, cudaStream_t st) {
  const int64_t blocks = (d.D + 127) / 128;
  k_glr_prefill<T><<<(unsigned)(blocks * d.b), 128, 0, st>>>(x, r, i, A, init, h, final_state, d, (int)blocks);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_glr_decode_step(float *state, const T *x, const T *r, const T *i, const float *A, T *h,
                                   const GlrDims &d, cudaStream_t st) {
  const int64_t blocks = (d.D + 127) / 128;
  k_glr_decode<T><<<(unsigned)(blocks * d.b), 128, 0, st>>>(state, x, r, i, A, h, d, (int)blocks);
  return cudaGetLastError();
}

size_t glr_backward_floats(const GlrDims &d) { return (size_t)d.b * d.D; }

template <typename T>
cudaError_t launch_glr_backward(const T *x, const T *r, const T *i, const float *A, const float *init, const T *h,
                                const T *dh, const float *dfinal, T *dx, T *dr, T *di, float *dA, float *dinit,
                                float *part, const GlrDims &d, cudaStream_t st) {
  const int64_t blocks = (d.D + 127) / 128;
  k_glr_backward<T><<<(unsigned)(blocks * d.b), 128, 0, st>>>(x, r, i, A, init, h, dh, dfinal, dx, dr, di, dinit, part,
                                                              d, (int)blocks);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_glr_sum<<<(unsigned)blocks, 128, 0, st>>>(part, dA, d.D, d.b);
  return cudaGetLastError();
}

#define SSD_GLR_INSTANCES(T)                                                                                           \
  template cudaError_t launch_glr_prefill<T>(const T *, const T *, const T *, const float *, const float *, T *,       \
                                             float *, const GlrDims &, cudaStream_t);                                  \
  template cudaError_t launch_glr_decode_step<T>(float *, const T *, const T *, const T *, const float *, T *,         \
                                                 const GlrDims &, cudaStream_t);                                       \
  template cudaError_t launch_glr_backward<T>(const T *, const T *, const T *, const float *, const float *, const T *, \
                                              const T *, const float *, T *, T *, T *, float *, float *, float *,      \
                                              const GlrDims &, cudaStream_t);
SSD_GLR_INSTANCES(float)
SSD_GLR_INSTANCES(__nv_bfloat16)

}  // namespace ssd
