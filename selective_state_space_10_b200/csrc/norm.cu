// norm.cu -- the norms around a mixer and their gradients: the residual norm before it (residual add, scale of the
// branch, RMS norm) and the gated norm after it (silu gate, RMS norm over each group of channels).  Statistics and
// sums over rows are fp32.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace ssd {

namespace {

constexpr int kThreads = 256;
constexpr int kParts = 592;  // most rows of partial sums

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

// Rows too long for registers.  One CTA per (row, group): a pass for the mean square, one that writes.
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

// Rows in registers.  A unit (one group of one row) belongs to `tpr` threads: a power of two up
// to a warp, with several units a CTA, or a whole CTA of tpr threads.  A thread holds NV runs of
// VEC neighbouring channels, so the row is read once, with 16-byte loads where the arrays allow.
template <int VEC, typename T>
__device__ __forceinline__ void load_run(const T *p, float (&v)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(q[k] << 16);
      v[2 * k + 1] = __uint_as_float(q[k] & 0xffff0000u);
    }
  } else if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int k = 0; k < VEC; k += 4) {
      const float4 u = load4(p + k);
      v[k] = u.x, v[k + 1] = u.y, v[k + 2] = u.z, v[k + 3] = u.w;
    }
  } else {
    v[0] = to_f32(p[0]);
  }
}
template <int VEC, typename T>
__device__ __forceinline__ void store_run(T *p, const float (&v)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 2) {
    uint4 u;
    uint32_t *q = &u.x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
      q[k] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = u;
  } else if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int k = 0; k < VEC; k += 4) *reinterpret_cast<float4 *>(p + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
  } else {
    p[0] = from_f32<T>(v[0]);
  }
}

// Sums over a unit's threads, in every one of them; all of the CTA's threads call it.  sh: N floats a warp.
template <int N>
__device__ __forceinline__ void unit_sum(float (&v)[N], int tpr, float *sh) {
  for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (tpr <= 32) return;
  __syncthreads();
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) sh[(threadIdx.x >> 5) * N + k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.f;
  const int first = threadIdx.x / tpr * (tpr >> 5);
  for (int j = first; j < first + (tpr >> 5); ++j)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += sh[j * N + k];
}

template <Mode M, typename TX, typename TR, int VEC, int NV>
__global__ void __launch_bounds__(1024)
    k_norm_rows(const TX *x, const float *__restrict__ scale, const TR *wide, const float *__restrict__ w, float eps,
                TR *wide_out, TX *out, NormDims d, int tpr, int W) {
  __shared__ float sh[32];
  const int lane = threadIdx.x % tpr;
  const int64_t unit = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = unit < d.rows * d.G;
  const int64_t row = live ? unit / d.G : 0;
  const int c0 = (int)(live ? unit % d.G : 0) * W;
  const TX *xr = x + row * (M == kResidual ? d.D : d.gate) + c0;
  const TR *wr = wide + row * d.D + c0;
  float v[NV][VEC], gate[M == kNormFirst ? NV : 1][VEC], ss[1] = {0.f};
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * tpr + lane) * VEC;
    if (!live || c >= W) continue;
    float a[VEC], b[VEC];
    load_run<VEC>(xr + c, a);
    if (M != kResidual || wide != nullptr) load_run<VEC>(wr + c, b);
    if (M == kResidual) {
      if (scale != nullptr) {
        float sc[VEC];
        load_run<VEC>(scale + c, sc);
#pragma unroll
        for (int e = 0; e < VEC; ++e) a[e] *= sc[e];
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[k][e] = wide != nullptr ? a[e] + b[e] : a[e];
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float g = a[e] * sigmoid(a[e]);
        v[k][e] = M == kGateFirst ? b[e] * g : b[e];
        if (M == kNormFirst) gate[k][e] = g;
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) ss[0] = fmaf(v[k][e], v[k][e], ss[0]);
  }
  unit_sum(ss, tpr, sh);
  const float rstd = rsqrtf(ss[0] / (float)W + eps);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * tpr + lane) * VEC;
    if (!live || c >= W) continue;
    if (M == kResidual && wide_out != nullptr) store_run<VEC>(wide_out + row * d.D + c0 + c, v[k]);
    float o[VEC];
    load_run<VEC>(w + c0 + c, o);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      o[e] *= v[k][e] * rstd;
      if (M == kNormFirst) o[e] *= gate[k][e];
    }
    store_run<VEC>(out + row * d.D + c0 + c, o);
  }
}

// Gradients of rows too long for registers.  A CTA takes rows blockIdx.x, + gridDim.x, ...; a column belongs to one thread of it, which adds the
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

// Gradients with rows in registers.  A CTA takes one group of channels and every P-th batch of `subs` rows, tpr
// threads a row (as k_norm_rows), and keeps its threads' sums over rows in registers.  Few CTAs hold such sums,
// so the loads of the rows to come are kept in flight by a ring of `stages` in shared memory: each thread copies
// there what itself will read, so no barrier guards it.  VEC = 1 (arrays without 16-byte alignment) loads
// directly.
__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void commit_async() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void wait_async(int left) {  // at most `left` (0 .. 3) groups still in flight
  if (left == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (left == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (left == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

constexpr int kRingBytes = 200 * 1024;  // of an SM's shared memory, all its CTAs together

// 16-byte pieces of a run of VEC channels of the four inputs
template <Mode M, typename TX, typename TR, int VEC>
struct Pieces {
  static constexpr int kX = VEC * (int)sizeof(TX) / 16, kR = VEC * (int)sizeof(TR) / 16;
  static constexpr int wide = 0, dout = kR, x = kR + kX, dwide = kR + 2 * kX;
  static constexpr int all = M == kResidual ? 2 * kR + 2 * kX : kR + 2 * kX;
};

template <Mode M, typename TX, typename TR, int VEC, int NV>
__global__ void __launch_bounds__(VEC *NV == 8 ? 640 : 512)
    k_norm_backward_rows(const TX *__restrict__ x, const float *__restrict__ scale, const TR *__restrict__ wide,
                         const float *__restrict__ w, float eps, const TX *__restrict__ dout, const TR *dwide, TX *dx,
                         TR *dwide_out, float *__restrict__ pw, float *__restrict__ ps, NormDims d, int tpr, int W,
                         int parts, int stages) {
  extern __shared__ __align__(16) char raw[];
  __shared__ float sh[2 * 32];
  using P = Pieces<M, TX, TR, VEC>;
  const int lane = threadIdx.x % tpr, sub = threadIdx.x / tpr, subs = blockDim.x / tpr;
  const int part = blockIdx.x % parts, c0 = blockIdx.x / parts * W;
  const int64_t step = (int64_t)parts * subs, first = (int64_t)part * subs;
  const int64_t turns = (d.rows - first + step - 1) / step;  // the same for all of the CTA
  const int64_t xs = M == kResidual ? d.D : d.gate;
  const bool want_x = M != kResidual || ps != nullptr, want_d = M == kResidual && dwide != nullptr;
  uint4 *ring = reinterpret_cast<uint4 *>(raw) + threadIdx.x;
  auto slot = [&](int stage, int k, int piece) { return ring + ((stage * NV + k) * P::all + piece) * blockDim.x; };
  auto fetch = [&](int64_t turn, int stage) {
    if constexpr (VEC > 1) {
      const int64_t row = first + turn * step + sub;
      if (turn < turns && row < d.rows)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int c = (k * tpr + lane) * VEC;
          if (c >= W) continue;
          const int64_t o = row * d.D + c0 + c;
#pragma unroll
          for (int q = 0; q < P::kR; ++q) {
            copy16(slot(stage, k, P::wide + q), reinterpret_cast<const uint4 *>(wide + o) + q);
            if (want_d) copy16(slot(stage, k, P::dwide + q), reinterpret_cast<const uint4 *>(dwide + o) + q);
          }
#pragma unroll
          for (int q = 0; q < P::kX; ++q) {
            copy16(slot(stage, k, P::dout + q), reinterpret_cast<const uint4 *>(dout + o) + q);
            if (want_x) copy16(slot(stage, k, P::x + q), reinterpret_cast<const uint4 *>(x + row * xs + c0 + c) + q);
          }
        }
      commit_async();
    }
  };
  // a run of one input, from the ring or from memory
  auto read = [&](int stage, int k, int piece, const auto *p, float (&v)[VEC]) {
    using T = std::remove_cv_t<std::remove_pointer_t<decltype(p)>>;
    if constexpr (VEC > 1) {
      constexpr int E = 16 / (int)sizeof(T);
#pragma unroll
      for (int q = 0; q < VEC / E; ++q) {
        float part[E];
        load_run<E>(reinterpret_cast<const T *>(slot(stage, k, piece + q)), part);
#pragma unroll
        for (int e = 0; e < E; ++e) v[q * E + e] = part[e];
      }
    } else {
      load_run<VEC>(p, v);
    }
  };
  float sw[NV][VEC], ss[M == kResidual ? NV : 1][VEC];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      sw[k][e] = 0.f;
      if (M == kResidual) ss[k][e] = 0.f;
    }
  for (int s = 0; s < stages; ++s) fetch(s, s);
  int stage = 0;
  for (int64_t turn = 0; turn < turns; ++turn) {
    const int64_t row = first + turn * step + sub, o = row * d.D + c0;
    const bool live = row < d.rows;
    if (VEC > 1) wait_async(stages - 1);
    // what is normed, the gradient of the weighted norm, its product with the weight, and the other inputs
    float v[NV][VEC], un[NV][VEC], uw[NV][VEC], other[NV][VEC], more[NV][VEC], sums[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * tpr + lane) * VEC;
      if (!live || c >= W) continue;
      read(stage, k, P::wide, wide + o + c, v[k]);
      read(stage, k, P::dout, dout + o + c, un[k]);
      if (want_x) read(stage, k, P::x, x + row * xs + c0 + c, other[k]);
      if (want_d) read(stage, k, P::dwide, dwide + o + c, more[k]);
      load_run<VEC>(w + c0 + c, uw[k]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (M == kGateFirst) {
          more[k][e] = v[k][e];  // y
          v[k][e] *= other[k][e] * sigmoid(other[k][e]);
        }
        if (M == kNormFirst) {
          more[k][e] = un[k][e];  // dout
          un[k][e] *= other[k][e] * sigmoid(other[k][e]);
        }
        uw[k][e] *= un[k][e];
        sums[0] = fmaf(v[k][e], v[k][e], sums[0]);
        sums[1] = fmaf(uw[k][e], v[k][e], sums[1]);
      }
    }
    fetch(turn + stages, stage);
    stage = stage + 1 == stages ? 0 : stage + 1;
    unit_sum(sums, tpr, sh);
    const float rstd = rsqrtf(sums[0] / (float)W + eps), mean = sums[1] * rstd / (float)W;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * tpr + lane) * VEC;
      if (!live || c >= W) continue;
      float a[VEC], b[VEC];
      if (M == kResidual && scale != nullptr) load_run<VEC>(scale + c, a);
      if (M == kNormFirst) load_run<VEC>(w + c0 + c, a);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float n = v[k][e] * rstd;
        float dv = rstd * (uw[k][e] - n * mean);
        sw[k][e] = fmaf(un[k][e], n, sw[k][e]);
        if (M == kResidual) {
          if (want_d) dv += more[k][e];
          if (ps != nullptr) ss[k][e] = fmaf(dv, other[k][e], ss[k][e]);
          a[e] = scale != nullptr ? dv * a[e] : dv;
          b[e] = dv;
        } else {
          const float z = other[k][e], sg = sigmoid(z), slope = sg * (1.f + z * (1.f - sg));
          a[e] = M == kGateFirst ? dv * more[k][e] * slope : more[k][e] * n * a[e] * slope;
          b[e] = M == kGateFirst ? dv * z * sg : dv;
        }
      }
      if (dx != nullptr) store_run<VEC>(dx + row * (M == kResidual ? d.D : d.dgate) + c0 + c, a);
      if (dwide_out != nullptr) store_run<VEC>(dwide_out + o + c, b);
    }
  }
  // the CTA's sums: over its units in order, through shared memory where there are several
  if (VEC > 1) wait_async(0);
  float *all = reinterpret_cast<float *>(raw);
  auto put = [&](float (&v)[NV][VEC], float *to) {
    if (subs > 1) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) all[(k * VEC + e) * blockDim.x + threadIdx.x] = v[k][e];
      __syncthreads();
      if (sub > 0) return;
      for (int u = 1; u < subs; ++u)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[k][e] += all[(k * VEC + e) * blockDim.x + u * tpr + lane];
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * tpr + lane) * VEC;
      if (c < W) store_run<VEC>(to + (int64_t)part * d.D + c0 + c, v[k]);
    }
  };
  if (pw != nullptr) put(sw, pw);
  if constexpr (M == kResidual)
    if (ps != nullptr) put(ss, ps);
}

// The partial sums of one or two vectors: 16 threads a column add every 16th, then one adds those, in order.
__global__ void __launch_bounds__(512) k_norm_sum(const float *__restrict__ pw, const float *__restrict__ ps, float *dw,
                                                  float *ds, int64_t D, int n) {
  __shared__ float sh[16][33];
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x % 32;
  const float *p = blockIdx.y == 0 ? pw : ps;
  float *o = blockIdx.y == 0 ? dw : ds;
  if (o == nullptr) return;
  float s = 0.f;
  if (c < D)
#pragma unroll 4
    for (int k = threadIdx.x / 32; k < n; k += 16) s += p[k * D + c];
  sh[threadIdx.x / 32][threadIdx.x % 32] = s;
  __syncthreads();
  if (threadIdx.x < 32 && c < D) {
    s = 0.f;
    for (int k = 0; k < 16; ++k) s += sh[k][threadIdx.x];
    o[c] = s;
  }
}

int parts_of(const NormDims &d) { return (int)std::min<int64_t>(d.rows, kParts); }

bool wide_ptr(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Threads a unit of n runs and runs a thread (1, 2 or 4); nv = 0: too many for registers.  Up to 32 runs, a
// power of two of lanes with one each; else whole warps, with the fewest idle lanes, and as many runs a thread
// as that allows.
struct Split {
  int tpr, nv;
};
Split split_unit(int64_t n, int most) {
  if (n <= 32) {
    int t = 1;
    while (t < n) t *= 2;
    return {t, 1};
  }
  Split best = {0, 0};
  int64_t idle = INT64_MAX;
  for (int nv = most; nv > 0; nv /= 2) {
    const int64_t t = ((n + nv - 1) / nv + 31) / 32 * 32;
    if (t <= 1024 && t * nv - n < idle) best = {(int)t, nv}, idle = t * nv - n;
  }
  return best;
}

template <Mode M, typename TX, typename TR, int VEC>
bool norm_rows(const TX *x, const float *scale, const TR *wide, const float *w, float eps, TR *wide_out, TX *out,
               const NormDims &d, cudaStream_t st) {
  const int64_t W = d.D / d.G;
  const Split p = split_unit((W + VEC - 1) / VEC, M == kNormFirst ? 2 : 4);
  if (p.nv == 0) return false;
  const int threads = p.tpr <= 32 ? 128 : p.tpr, units = threads / p.tpr;
  const unsigned grid = (unsigned)((d.rows * d.G + units - 1) / units);
  auto run = [&](auto *f) { f<<<grid, threads, 0, st>>>(x, scale, wide, w, eps, wide_out, out, d, p.tpr, (int)W); };
  if (p.nv == 4) run(k_norm_rows<M, TX, TR, VEC, 4>);
  else if (p.nv == 2) run(k_norm_rows<M, TX, TR, VEC, 2>);
  else run(k_norm_rows<M, TX, TR, VEC, 1>);
  return true;
}

template <Mode M, typename TX, typename TR>
cudaError_t norm(const TX *x, const float *scale, const TR *wide, const float *w, float eps, TR *wide_out, TX *out,
                 const NormDims &d, cudaStream_t st) {
  constexpr int VEC = sizeof(TX) == 2 ? 8 : 4;
  const bool vec = (d.D / d.G) % VEC == 0 && d.gate % VEC == 0 && wide_ptr(x) && wide_ptr(scale) && wide_ptr(wide) &&
                   wide_ptr(w) && wide_ptr(wide_out) && wide_ptr(out);
  if (!(vec ? norm_rows<M, TX, TR, VEC>(x, scale, wide, w, eps, wide_out, out, d, st)
            : norm_rows<M, TX, TR, 1>(x, scale, wide, w, eps, wide_out, out, d, st)))
    k_norm<M, TX, TR><<<(unsigned)(d.rows * d.G), kThreads, 0, st>>>(x, scale, wide, w, eps, wide_out, out, d);
  return cudaGetLastError();
}

// Runs the register kernel and sets `parts`; false: rows too long for it.
template <Mode M, typename TX, typename TR, int VEC, int NV>
bool norm_backward_rows(const TX *x, const float *scale, const TR *wide, const float *w, float eps, const TX *dout,
                        const TR *dwide, TX *dx, TR *dwide_out, float *pw, float *ps, const NormDims &d, int &parts,
                        cudaError_t &err, cudaStream_t st) {
  const int64_t W = d.D / d.G, n = (W + VEC - 1) / VEC;
  constexpr int most = VEC * NV == 8 ? 640 : 512;
  const int64_t t = n <= 32 ? split_unit(n, 1).tpr : ((n + NV - 1) / NV + 31) / 32 * 32;
  if (t > most) return false;
  const int tpr = (int)t, subs = std::max(1, 256 / tpr), threads = subs * tpr;
  const int resident = std::max(1, most / threads);
  parts = (int)std::max<int64_t>(1, std::min<int64_t>({(d.rows + subs - 1) / subs, 148 * resident / d.G, parts}));
  const int stage = VEC > 1 ? threads * NV * Pieces<M, TX, TR, VEC>::all * 16 : 0;
  const int stages = VEC > 1 ? std::max(1, std::min(4, kRingBytes / resident / stage)) : 1;
  const size_t smem = std::max((size_t)stages * stage, (size_t)threads * VEC * NV * 4);
  auto *f = k_norm_backward_rows<M, TX, TR, VEC, NV>;
  err = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return true;
  f<<<(unsigned)(parts * d.G), threads, smem, st>>>(x, scale, wide, w, eps, dout, dwide, dx, dwide_out, pw, ps, d, tpr,
                                                    (int)W, parts, stages);
  err = cudaGetLastError();
  return true;
}

template <Mode M, typename TX, typename TR>
cudaError_t norm_backward(const TX *x, const float *scale, const TR *wide, const float *w, float eps, const TX *dout,
                          const TR *dwide, TX *dx, TR *dwide_out, float *dw, float *ds, float *part, const NormDims &d,
                          cudaStream_t st) {
  int parts = parts_of(d);
  float *pw = dw != nullptr ? part : nullptr, *ps = ds != nullptr ? part + (int64_t)parts * d.D : nullptr;
  constexpr int VEC = sizeof(TX) == 2 ? 8 : 4;
  const bool vec = (d.D / d.G) % VEC == 0 && d.gate % VEC == 0 && d.dgate % VEC == 0 && wide_ptr(x) && wide_ptr(scale) &&
                   wide_ptr(wide) && wide_ptr(w) && wide_ptr(dout) && wide_ptr(dwide) && wide_ptr(dx) &&
                   wide_ptr(dwide_out);
  cudaError_t e = cudaSuccess;
  auto rows = [&](auto nv, auto v) {
    return norm_backward_rows<M, TX, TR, decltype(v)::value, decltype(nv)::value>(
        x, scale, wide, w, eps, dout, dwide, dx, dwide_out, pw, ps, d, parts, e, st);
  };
  bool done;
  if (vec)
    done = rows(std::integral_constant<int, 8 / VEC>{}, std::integral_constant<int, VEC>{}) ||
           rows(std::integral_constant<int, 16 / VEC>{}, std::integral_constant<int, VEC>{});
  else
    done = rows(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  if (!done) {
    k_norm_backward<M, TX, TR><<<parts, kThreads, 0, st>>>(x, scale, wide, w, eps, dout, dwide, dx, dwide_out, pw, ps, d);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || (dw == nullptr && ds == nullptr)) return e;
  k_norm_sum<<<dim3((unsigned)((d.D + 31) / 32), ds != nullptr ? 2 : 1), 512, 0, st>>>(pw, ps, dw, ds, d.D, parts);
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
