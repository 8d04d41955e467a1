// norm.cu -- the norms around a mixer and their gradients: the residual norm before it (residual add, scale of the
// branch, RMS norm) and the gated norm after it (silu gate, RMS norm over each group of channels).  Statistics and
// sums over rows are fp32.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace ssd {

namespace {

constexpr int kThreads = 256;
constexpr int kParts = 592;  // most rows of partial sums

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
// to a warp, with several units a CTA, or whole warps.  A thread holds NV runs of VEC neighbouring
// channels, run k at (k tpr + lane) VEC, so the row is read once, with 16-byte loads where the
// arrays allow (VEC = 1: element loads).  All loads are issued before the first use; runs past the
// unit's end are loaded from its start and set to zero.
// Most threads of a CTA whose threads hold n channels each.
constexpr int row_threads(int n) { return n > 16 ? 512 : 1024; }

template <typename T, int VEC, int NV>
struct Runs {
  static constexpr int kPieces = VEC > 1 ? VEC * (int)sizeof(T) / 16 : 1;  // 16-byte pieces a run
  using Piece = std::conditional_t<(VEC > 1), uint4, T>;
  Piece q[NV][kPieces];

  // from memory: run k at p + at[k]; kSectors: a run of 8 fp32 at once
  template <bool kSectors = false>
  __device__ __forceinline__ void load(const T *p, const int (&at)[NV]) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if constexpr (kSectors && VEC == 8 && sizeof(T) == 4) {
        ulonglong2 a, b;
        asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];" : "=l"(a.x), "=l"(a.y), "=l"(b.x), "=l"(b.y) : "l"(p + at[k]));
        q[k][0] = *reinterpret_cast<uint4 *>(&a);
        q[k][1] = *reinterpret_cast<uint4 *>(&b);
      } else {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) q[k][j] = reinterpret_cast<const Piece *>(p + at[k])[j];
      }
  }
  // from the thread's pieces in shared memory, `pitch` apart; those of a run begin `run` pieces after the last one's
  __device__ __forceinline__ void load_pieces(const uint4 *from, int run, int pitch) {
    if constexpr (VEC > 1)
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < kPieces; ++j) q[k][j] = from[(k * run + j) * pitch];
  }
  // the thread's channels 2 e and 2 e + 1, in the order of its runs
  __device__ __forceinline__ f2 operator[](int e) const {
    if constexpr (VEC == 1) {
      return mk(to_f32(q[2 * e][0]), to_f32(q[2 * e + 1][0]));
    } else {
      const int k = 2 * e / VEC, c = 2 * e % VEC, per = 16 / (int)sizeof(T);
      const uint4 &u = q[k][c / per];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      if constexpr (sizeof(T) == 2)
        return from_bf16x2(w[c % per / 2]);
      else
        return mk(__uint_as_float(w[c % per]), __uint_as_float(w[c % per + 1]));
    }
  }
};

// Out again, rounded; run k at p + at[k] where on[k].  Runs of 8 fp32 are whole 32-byte sectors, stored in one piece where
// the array is aligned to them (residual norm of 4096 x 2560: 21.8 us, 22.6 us in halves; gated gradient of 4096 x 5120: 66
// and 69 us).
template <typename T, int VEC, int NV, bool kSectors = true>
__device__ __forceinline__ void store_runs(T *p, const int (&at)[NV], const bool (&on)[NV], const f2 (&v)[NV * VEC / 2]) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (!on[k]) continue;
    if constexpr (VEC == 1) {
      const float2 s = split(v[k / 2]);
      p[at[k]] = from_f32<T>(k % 2 ? s.y : s.x);
    } else if constexpr (sizeof(T) == 2) {
      const f2 *e = &v[k * VEC / 2];
      *reinterpret_cast<uint4 *>(p + at[k]) =
          make_uint4(to_bf16x2(e[0]), to_bf16x2(e[1]), to_bf16x2(e[2]), to_bf16x2(e[3]));
    } else {
      const f2 *e = &v[k * VEC / 2];
      if constexpr (VEC == 8 && kSectors) {
        asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p + at[k]), "l"(e[0].v), "l"(e[1].v), "l"(e[2].v),
                     "l"(e[3].v)
                     : "memory");
      } else {
#pragma unroll
        for (int c = 0; c < VEC / 4; ++c)
          *reinterpret_cast<ulonglong2 *>(p + at[k] + 4 * c) = make_ulonglong2(e[2 * c].v, e[2 * c + 1].v);
      }
    }
  }
}

template <int VEC, int NV>
__device__ __forceinline__ void zero_off(f2 (&v)[NV * VEC / 2], const bool (&on)[NV]) {
#pragma unroll
  for (int e = 0; e < NV * VEC / 2; ++e) {
    const float2 s = split(v[e]);
    v[e] = mk(on[2 * e / VEC] ? s.x : 0.f, on[(2 * e + 1) / VEC] ? s.y : 0.f);
  }
}

__device__ __forceinline__ float total(f2 v) {
  const float2 s = split(v);
  return s.x + s.y;
}

__device__ __forceinline__ float from_lane(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

// The sum over a unit's threads, in every one of them; sh: one float a warp.  A unit of several warps is a whole CTA.
__device__ __forceinline__ float unit_sum(float v, int tpr, float *sh) {
  if (tpr < 32) {
    for (int o = tpr >> 1; o > 0; o >>= 1) v += from_lane(v, o);
    return v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += from_lane(v, o);
  if (tpr == 32) return v;
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh[0];
  for (int j = 1; j < (tpr >> 5); ++j) v += sh[j];
  return v;
}

// Two sums; sh: a pair a warp of the CTA, not used by the call before (two buffers in turn).  The units of several
// warps that share a CTA meet at barriers of their own (a kernel with numbered barriers takes all 16 of a CTA, and an SM
// has 64: no more than 4 CTAs fit).  Half a warp adds up each sum: one exchange in place of one for each.
__device__ __forceinline__ float2 unit_sums(float a, float b, int tpr, f2 *sh) {
  if (tpr < 32) {
    for (int o = tpr >> 1; o > 0; o >>= 1) a += from_lane(a, o), b += from_lane(b, o);
    return make_float2(a, b);
  }
  const bool upper = threadIdx.x & 16;
  float v = upper ? b : a;
  v += from_lane(upper ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += from_lane(v, o);
  if (tpr == 32) return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
  const int warps = tpr >> 5, unit = tpr == blockDim.x ? 0 : threadIdx.x / tpr;
  if ((threadIdx.x & 15) == 0) reinterpret_cast<float *>(sh)[threadIdx.x >> 4] = v;
  if (tpr == blockDim.x)
    __syncthreads();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(unit + 1), "r"(tpr) : "memory");
  f2 s = sh[unit * warps];
  for (int j = 1; j < warps; ++j) s = s + sh[unit * warps + j];
  return split(s);
}

// Bound by memory, with the loads of about 10 rows an SM in flight: residual norm of 4096 x 2560 (bf16 beside an fp32
// stream, 126 MB) 21.6 us, 5.8 TB/s, 89 % of the measured copy bandwidth; gated norm of 4096 x 5120 (fp32 y, 168 MB)
// 33.0 us, 5.1 TB/s, 78 %.
template <Mode M, typename TX, typename TR, int VEC, int NV>
__global__ void __launch_bounds__(row_threads(NV *VEC))
    k_norm_rows(const TX *x, const float *scale, const TR *wide, const float *w, float eps, TR *wide_out, TX *out,
                NormDims d, int tpr, int W) {
  __shared__ float sh[32];
  sm100::grid_dep_launch();
  sm100::grid_dep_wait();
  constexpr int E = NV * VEC / 2;
  const int lane = threadIdx.x % tpr;
  const int64_t unit = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = unit < d.rows * d.G;
  const int64_t row = live ? unit / d.G : 0;
  const int c0 = (int)(live ? unit % d.G : 0) * W;
  int at[NV];
  bool on[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    at[k] = (k * tpr + lane) * VEC;
    on[k] = live && at[k] < W;
    if (!on[k]) at[k] = 0;
  }
  Runs<TX, VEC, NV> rx;
  Runs<TR, VEC, NV> rw;
  rx.load(x + row * (M == kResidual ? d.D : d.gate) + c0, at);
  if (M != kResidual || wide != nullptr) rw.template load<true>(wide + row * d.D + c0, at);
  f2 v[E], gate[M == kNormFirst ? E : 1];
  if (M == kResidual) {
    if (scale != nullptr) {
      Runs<float, VEC, NV> rs;
      rs.load(scale, at);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = rx[e] * rs[e];
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = rx[e];
    }
    if (wide != nullptr)
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = v[e] + rw[e];
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const f2 z = rx[e], g = z * sigmoid(z);
      v[e] = M == kGateFirst ? rw[e] * g : rw[e];
      if (M == kNormFirst) gate[e] = g;
    }
  }
  if (!on[NV - 1]) zero_off<VEC, NV>(v, on);
  f2 ss = both(0.f);
#pragma unroll
  for (int e = 0; e < E; ++e) ss = fma2(v[e], v[e], ss);
  // The weights' loads pass the row's barrier where the gate follows the norm (bf16 beside fp32 y, 3276 x 5120: 25.7 us,
  // 27.9 us after it); elsewhere the registers that they hold cost as much or more.
  constexpr bool kEarly = M == kNormFirst && VEC > 1;
  Runs<float, VEC, NV> rg;
  if (kEarly) rg.load(w + c0, at);
  const f2 rstd = both(rsqrtf(unit_sum(total(ss), tpr, sh) / (float)W + eps));
  if (M == kResidual && wide_out != nullptr) store_runs<TR, VEC, NV>(wide_out + row * d.D + c0, at, on, v);
  if (!kEarly) rg.load(w + c0, at);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    v[e] = v[e] * rstd * rg[e];
    if (M == kNormFirst) v[e] = v[e] * gate[e];
  }
  store_runs<TX, VEC, NV>(out + row * d.D + c0, at, on, v);
}

// Gradients of rows too long for registers.  A CTA takes rows blockIdx.x, + gridDim.x, ...; a column belongs to one thread
// of it, which adds the row's terms to the CTA's partial sums.
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

// Gradients with rows in registers.  A CTA takes one group of channels and every `parts`-th batch of `subs` rows, tpr
// threads a row (as k_norm_rows), and keeps its threads' sums over rows in registers.  Few CTAs hold such sums,
// so the loads of the rows to come are kept in flight by a ring of `stages` in shared memory: each thread copies
// there what itself will read, so no barrier guards it.  A row's inputs are read from the ring twice, before and
// after its two sums are known, rather than held in registers.  VEC = 1 (arrays without 16-byte alignment) loads
// directly.
// Gated norm of 4096 x 5120 (bf16 beside fp32 y, 294 MB): 66 us with the sum of the partial rows, 4.4 TB/s, 68 % of the
// measured copy bandwidth; residual norm of 65536 x 768 (906 MB) 200 us, 4.5 TB/s, 69 %.  Bound first by reads of shared
// memory (the ring twice, the weights again for every row: the most frequent stall), then by each row's own chain (ring,
// sums, ring, stores) on the 24 warps an SM that the sums' registers leave: issue slots 42 % busy.
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
// Threads of an SM, all its CTAs together, which leaves each 80 registers (43690 x 768 bf16 beside fp32, gated and
// residual: 96 and 118 us; 640 threads 102 and 123, 896 threads 97 and 119; at 2560 and 5120 channels 640 and 768 run
// alike, 896 up to 15 % longer).
constexpr int kRowThreads = 768;

// 16-byte pieces of a run of VEC channels of the four inputs, and of an fp32 vector
template <Mode M, typename TX, typename TR, int VEC>
struct Pieces {
  enum : int {
    kX = VEC * (int)sizeof(TX) / 16, kR = VEC * (int)sizeof(TR) / 16, kF = VEC / 4,
    wide = 0, dout = kR, x = kR + kX, dwide = kR + 2 * kX,  // where each input's pieces begin
    all = M == kResidual ? 2 * kR + 2 * kX : kR + 2 * kX
  };
};

template <Mode M, typename TX, typename TR, int VEC, int NV>
__device__ __forceinline__ void backward_rows(const TX *x, const float *scale, const TR *wide, const float *w, float eps,
                                              const TX *dout, const TR *dwide, TX *dx, TR *dwide_out, float *pw, float *ps,
                                              const NormDims &d, int tpr, int W, int parts, int stages) {
  extern __shared__ __align__(16) char raw[];
  __shared__ f2 sh[2][32];
  using P = Pieces<M, TX, TR, VEC>;
  constexpr int E = NV * VEC / 2;
  const int lane = threadIdx.x % tpr, sub = threadIdx.x / tpr, subs = blockDim.x / tpr;
  const int part = blockIdx.x % parts, c0 = blockIdx.x / parts * W;
  const unsigned rows = (unsigned)d.rows, step = parts * subs, first = part * subs;  // rows < 2^31
  const int turns = (int)((rows - first + step - 1) / step);                          // the same for all of the CTA
  const int D = (int)d.D;
  const int64_t xs = M == kResidual ? D : d.gate;
  const float per = 1.f / (float)W;
  const bool want_x = M != kResidual || ps != nullptr, want_d = M == kResidual && dwide != nullptr;
  int at[NV];
  bool in[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    at[k] = (k * tpr + lane) * VEC;
    in[k] = at[k] < W;
    if (!in[k]) at[k] = 0;
  }
  // a thread's pieces lie blockDim.x apart, so that a warp's accesses are contiguous
  const int pitch = blockDim.x, stage_pitch = NV * P::all * pitch;
  const bool scaled = M == kResidual && scale != nullptr;
  uint4 *ring = reinterpret_cast<uint4 *>(raw) + threadIdx.x;
  uint4 *mine = ring + stages * stage_pitch;  // this thread's weights (and scales), behind the ring
  unsigned ahead = first + sub;  // the next row to fetch
  auto fetch = [&](int stage) {
    if constexpr (VEC > 1) {
      const unsigned row = ahead;
      ahead = min(ahead + step, 0x80000000u);
      if (row < rows) {
        const int64_t o = (int64_t)row * D + c0;
        uint4 *slot = ring + stage * stage_pitch;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          uint4 *to = slot + k * P::all * pitch;
#pragma unroll
          for (int q = 0; q < P::kR; ++q) {
            copy16(to + (P::wide + q) * pitch, reinterpret_cast<const uint4 *>(wide + o + at[k]) + q);
            if (want_d) copy16(to + (P::dwide + q) * pitch, reinterpret_cast<const uint4 *>(dwide + o + at[k]) + q);
          }
#pragma unroll
          for (int q = 0; q < P::kX; ++q) {
            copy16(to + (P::dout + q) * pitch, reinterpret_cast<const uint4 *>(dout + o + at[k]) + q);
            if (want_x)
              copy16(to + (P::x + q) * pitch, reinterpret_cast<const uint4 *>(x + row * xs + c0 + at[k]) + q);
          }
        }
      }
      commit_async();
    }
  };
  if constexpr (VEC > 1)
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int q = 0; q < P::kF; ++q) {
        mine[(k * P::kF + q) * pitch] = reinterpret_cast<const uint4 *>(w + c0 + at[k])[q];
        if (scaled) mine[((NV + k) * P::kF + q) * pitch] = reinterpret_cast<const uint4 *>(scale + at[k])[q];
      }
  f2 sw[E], ss[M == kResidual ? E : 1];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    sw[e] = both(0.f);
    if (M == kResidual) ss[e] = both(0.f);
  }
  for (int s = 0; s < stages; ++s) fetch(s);
  int stage = 0;
  unsigned row = first + sub;
  for (int turn = 0; turn < turns; ++turn, row += step) {
    const bool live = row < rows;
    bool on[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) on[k] = live && in[k];
    if constexpr (VEC > 1) wait_async(stages - 1);
    const uint4 *slot = ring + stage * stage_pitch;
    // a run of an input: from its slot, each time it is needed, or from memory
    auto weight = [&](auto &runs, int vector, const float *p) {
      if constexpr (VEC > 1) runs.load_pieces(mine + vector * NV * P::kF * pitch, P::kF, pitch);
      else runs.load(p, at);
    };
    auto take = [&](auto &runs, int piece, const auto *p) {
      if constexpr (VEC > 1) runs.load_pieces(slot + piece * pitch, P::all, pitch);
      else runs.load(p, at);
    };
    const unsigned r = live ? row : 0;
    const int64_t ro = (int64_t)r * D + c0;
    // v: what is normed; uw: the gradient of the weighted norm times the weight
    f2 v[E], uw[E], s0 = both(0.f), s1 = both(0.f);
    {
      Runs<TR, VEC, NV> rwide;
      Runs<TX, VEC, NV> rdout, rx;
      Runs<float, VEC, NV> rg;
      take(rwide, P::wide, wide + ro);
      take(rdout, P::dout, dout + ro);
      if (M != kResidual) take(rx, P::x, x + r * xs + c0);
      weight(rg, 0, w + c0);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[e] = rwide[e];
        uw[e] = rdout[e] * rg[e];
        if (M != kResidual) {
          const f2 z = rx[e], g = z * sigmoid(z);
          if (M == kGateFirst) v[e] = v[e] * g;
          if (M == kNormFirst) uw[e] = uw[e] * g;
        }
      }
    }
    if (!on[NV - 1]) {
      zero_off<VEC, NV>(v, on);
      zero_off<VEC, NV>(uw, on);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      s0 = fma2(v[e], v[e], s0);
      s1 = fma2(uw[e], v[e], s1);
    }
    const float2 sums = unit_sums(total(s0), total(s1), tpr, sh[turn & 1]);
    if (live) {  // nothing was fetched for a row past the last one
      const float rs1 = rsqrtf(fmaf(sums.x, per, eps));
      const f2 rstd = both(rs1), mean = both(-sums.y * rs1 * per);
      Runs<TX, VEC, NV> rdout, rx;
      f2 a[E];
      take(rdout, P::dout, dout + ro);
      if (want_x) take(rx, P::x, x + r * xs + c0);
      if (M == kResidual) {
        Runs<float, VEC, NV> rs;
        Runs<TR, VEC, NV> rd;
        if (want_d) take(rd, P::dwide, dwide + ro);
        if (scaled) weight(rs, 1, scale);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const f2 n = v[e] * rstd;
          f2 dv = rstd * fma2(n, mean, uw[e]);
          sw[e] = fma2(rdout[e], n, sw[e]);
          if (want_d) dv = dv + rd[e];
          if (ps != nullptr) ss[e] = fma2(dv, rx[e], ss[e]);
          a[e] = scaled ? dv * rs[e] : dv;
          v[e] = dv;
        }
      } else {
        Runs<TR, VEC, NV> ry;
        Runs<float, VEC, NV> rg;
        if (M == kGateFirst) take(ry, P::wide, wide + ro);
        if (M == kNormFirst) weight(rg, 0, w + c0);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const f2 n = v[e] * rstd, z = rx[e], sg = sigmoid(z), g = z * sg;
          const f2 dv = rstd * fma2(n, mean, uw[e]), slope = fma2(g, fma2(sg, both(-1.f), both(1.f)), sg);
          if (M == kGateFirst) {
            sw[e] = fma2(rdout[e], n, sw[e]);
            a[e] = dv * ry[e] * slope;
            v[e] = dv * g;
          } else {
            sw[e] = fma2(rdout[e] * g, n, sw[e]);
            a[e] = rdout[e] * rg[e] * n * slope;
            v[e] = dv;
          }
        }
      }
      if (dx != nullptr) store_runs<TX, VEC, NV>(dx + row * (M == kResidual ? (int64_t)D : d.dgate) + c0, at, on, a);
      if (dwide_out != nullptr) store_runs<TR, VEC, NV>(dwide_out + ro, at, on, v);
    }
    fetch(stage);
    stage = stage + 1 == stages ? 0 : stage + 1;
  }
  // the CTA's sums: over its units in order, through shared memory where there are several
  if (VEC > 1) wait_async(0);
  f2 *all = reinterpret_cast<f2 *>(raw);
  auto put = [&](f2 (&v)[E], float *to) {
    if (subs > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < E; ++e) all[e * blockDim.x + threadIdx.x] = v[e];
      __syncthreads();
      if (sub > 0) return;
      for (int u = 1; u < subs; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = v[e] + all[e * blockDim.x + u * tpr + lane];
    }
    store_runs<float, VEC, NV, false>(to + (int64_t)part * d.D + c0, at, in, v);  // a workspace has 16-byte alignment
  };
  if (pw != nullptr) put(sw, pw);
  if constexpr (M == kResidual)
    if (ps != nullptr) put(ss, ps);
}

template <Mode M, typename TX, typename TR, int VEC, int NV>
__global__ void __launch_bounds__(kRowThreads)
    k_norm_backward_rows(const TX *x, const float *scale, const TR *wide, const float *w, float eps, const TX *dout,
                         const TR *dwide, TX *dx, TR *dwide_out, float *pw, float *ps, NormDims d, int tpr, int W, int parts,
                         int stages) {
  sm100::grid_dep_wait();
  backward_rows<M, TX, TR, VEC, NV>(x, scale, wide, w, eps, dout, dwide, dx, dwide_out, pw, ps, d, tpr, W, parts, stages);
}

// VEC = 1.  Not launched early, so that the pointers may be __restrict__: its loads, unlike the ring's copies, then pass
// the row's barrier and stores (bf16, 10922 x 1537, gates after the norm: 80.7 us, 93.0 us without).
template <Mode M, typename TX, typename TR, int NV>
__global__ void __launch_bounds__(kRowThreads)
    k_norm_backward_elements(const TX *__restrict__ x, const float *__restrict__ scale, const TR *__restrict__ wide,
                             const float *__restrict__ w, float eps, const TX *__restrict__ dout, const TR *dwide, TX *dx,
                             TR *dwide_out, float *__restrict__ pw, float *__restrict__ ps, NormDims d, int tpr, int W,
                             int parts, int stages) {
  backward_rows<M, TX, TR, 1, NV>(x, scale, wide, w, eps, dout, dwide, dx, dwide_out, pw, ps, d, tpr, W, parts, stages);
}

// The partial sums of one or two vectors, n rows of D: 32 threads a column add every 32nd row, then a warp adds those.
__global__ void __launch_bounds__(1024) k_row_sums(const float *p0, const float *p1, float *o0, float *o1,
                                                   int64_t D, int64_t n) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32;
  const float *p = blockIdx.y == 0 ? p0 : p1;
  float *o = blockIdx.y == 0 ? o0 : o1;
  sm100::grid_dep_wait();  // for the partial sums
  if (o == nullptr) return;
  float s = 0.f;
  if (c + lane < D)
#pragma unroll 8
    for (int64_t j = warp; j < n; j += 32) s += p[j * D + c + lane];
  sh[warp][lane] = s;
  __syncthreads();
  s = warp_sum(sh[lane][warp], 32);
  if (lane == 0 && c + warp < D) o[c + warp] = s;
}

int parts_of(const NormDims &d) { return (int)std::min<int64_t>(d.rows, kParts); }

// A run of 8 bf16 or 4 fp32 takes 16-byte alignment, a run of 8 fp32, which is stored in one piece, 32.
template <typename T>
bool wide_ptr(const T *p, int channels) {
  return reinterpret_cast<uintptr_t>(p) % (sizeof(T) * channels) == 0;
}

// Threads a unit of n runs and runs a thread (least .. most, powers of two); nv = 0: too many for registers.  Up
// to 32 least runs, a power of two of lanes; else whole warps, with the most runs a thread that leave no more than an
// eighth of the lanes' runs idle (a quarter for runs of one channel), or else those that leave the fewest.  Forward,
// fp32, groups of 1920: 4 runs with 6 % idle 60 us, 1 with none 89 us; bf16 beside fp32, 4096 x 2560: 2 with none idle
// 21.6 us, 4 with 17 % 24.4 us; bf16, 16384 x 1537: 8 single channels with 14 % 79 us, 2 with 4 % 148 us.  limit(nv): the
// most threads of a CTA.
struct Split {
  int tpr, nv;
};
template <typename F>
Split split_unit(int64_t n, int least, int most, F limit) {
  if (n <= 32 * least) {
    int t = 1;
    while (t * least < n) t *= 2;
    return {t, least};
  }
  Split best = {0, 0};
  int64_t idle = INT64_MAX;
  for (int nv = most; nv >= least; nv /= 2) {
    const int64_t t = ((n + nv - 1) / nv + 31) / 32 * 32;
    if (t <= limit(nv) && t * nv - n < idle) best = {(int)t, nv}, idle = t * nv - n;
    if (best.nv > 0 && idle * (least == 2 ? 4 : 8) <= (int64_t)best.tpr * best.nv) break;
  }
  return best;
}

template <Mode M, typename TX, typename TR, int VEC>
bool norm_rows(const TX *x, const float *scale, const TR *wide, const float *w, float eps, TR *wide_out, TX *out,
               const NormDims &d, cudaError_t &err, cudaStream_t st) {
  const int64_t W = d.D / d.G;
  constexpr int least = VEC == 1 ? 2 : 1;
  const Split p = split_unit((W + VEC - 1) / VEC, least, 4 * least, [](int nv) { return row_threads(nv * VEC); });
  if (p.nv == 0) return false;
  const int threads = p.tpr <= 32 ? 128 : p.tpr, units = threads / p.tpr;
  const unsigned grid = (unsigned)((d.rows * d.G + units - 1) / units);
  auto run = [&](auto *f) {
    err = launch_dependent(f, grid, threads, 0, st, x, scale, wide, w, eps, wide_out, out, d, p.tpr, (int)W);
  };
  if (p.nv == 4 * least) run(k_norm_rows<M, TX, TR, VEC, 4 * least>);
  else if (p.nv == 2 * least) run(k_norm_rows<M, TX, TR, VEC, 2 * least>);
  else run(k_norm_rows<M, TX, TR, VEC, least>);
  return true;
}

template <Mode M, typename TX, typename TR>
cudaError_t norm(const TX *x, const float *scale, const TR *wide, const float *w, float eps, TR *wide_out, TX *out,
                 const NormDims &d, cudaStream_t st) {
  constexpr int VEC = sizeof(TX) == 2 ? 8 : 4;
  const bool vec = (d.D / d.G) % VEC == 0 && d.gate % VEC == 0 && wide_ptr(x, VEC) && wide_ptr(scale, 4) && wide_ptr(wide, VEC) &&
                   wide_ptr(w, 4) && wide_ptr(wide_out, VEC) && wide_ptr(out, VEC);
  cudaError_t err = cudaSuccess;
  if (vec ? norm_rows<M, TX, TR, VEC>(x, scale, wide, w, eps, wide_out, out, d, err, st)
          : norm_rows<M, TX, TR, 1>(x, scale, wide, w, eps, wide_out, out, d, err, st))
    return err;
  return launch(k_norm<M, TX, TR>, dim3((unsigned)(d.rows * d.G)), kThreads, 0, st, false, x, scale, wide, w, eps, wide_out,
                out, d);
}

// Most dynamic shared memory of a CTA: 227 KB but for the kernel's own arrays.
constexpr int kMaxSmem = 227 * 1024 - 512;

// Runs the register kernel and sets `parts`; false: rows too long for it, or for one stage of its ring beside the weights
// in the shared memory of a CTA (residual norm with 16 channels a thread: from 9220 fp32 channels with a scale, 11268
// without, 11272 bf16 ones beside fp32 with a scale).  The kernel for long rows takes those at about half the rate: 2048
// rows of bf16 beside fp32 with a scale, 11264 channels here 182 us, 12288 there 396 us.
template <Mode M, typename TX, typename TR, int VEC, int NV>
bool norm_backward_rows(const TX *x, const float *scale, const TR *wide, const float *w, float eps, const TX *dout,
                        const TR *dwide, TX *dx, TR *dwide_out, float *pw, float *ps, const NormDims &d, int &parts,
                        cudaError_t &err, cudaStream_t st) {
  const int64_t W = d.D / d.G, n = (W + VEC - 1) / VEC;
  const int tpr = split_unit(n, NV, NV, [](int) { return kRowThreads; }).tpr;
  if (tpr == 0) return false;
  const int subs = std::max(1, 256 / tpr), threads = subs * tpr;
  const int resident = std::max(1, kRowThreads / threads);
  using P = Pieces<M, TX, TR, VEC>;
  const int stage = VEC > 1 ? threads * NV * P::all * 16 : 0;
  const int fixed = VEC > 1 ? threads * NV * P::kF * 16 * (M == kResidual && scale != nullptr ? 2 : 1) : 0;
  const int stages = VEC > 1 ? std::max(1, std::min(4, (kRingBytes / resident - fixed) / stage)) : 1;
  const size_t smem = std::max((size_t)stages * stage + fixed, (size_t)threads * VEC * NV * 4);
  if (smem > kMaxSmem) return false;
  parts = (int)std::max<int64_t>(1, std::min<int64_t>({(d.rows + subs - 1) / subs, 148 * resident / d.G, parts}));
  const dim3 grid((unsigned)(parts * d.G));
  if constexpr (VEC > 1) {
    auto *f = k_norm_backward_rows<M, TX, TR, VEC, NV>;
    // the same limit in every call: another thread's call with a size of its own may come between this and the launch
    err = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (err == cudaSuccess)
      err = launch_dependent(f, grid, threads, smem, st, x, scale, wide, w, eps, dout, dwide, dx, dwide_out, pw, ps, d, tpr,
                             (int)W, parts, stages);
  } else {  // at most 24 KB
    err = launch(k_norm_backward_elements<M, TX, TR, NV>, grid, threads, smem, st, false, x, scale, wide, w, eps, dout, dwide,
                 dx, dwide_out, pw, ps, d, tpr, (int)W, parts, stages);
  }
  return true;
}

template <Mode M, typename TX, typename TR>
cudaError_t norm_backward(const TX *x, const float *scale, const TR *wide, const float *w, float eps, const TX *dout,
                          const TR *dwide, TX *dx, TR *dwide_out, float *dw, float *ds, float *part, const NormDims &d,
                          cudaStream_t st) {
  int parts = parts_of(d);
  float *pw = dw != nullptr ? part : nullptr, *ps = ds != nullptr ? part + (int64_t)parts * d.D : nullptr;
  constexpr int VEC = sizeof(TX) == 2 ? 8 : 4;
  const bool vec = (d.D / d.G) % VEC == 0 && d.gate % VEC == 0 && d.dgate % VEC == 0 && wide_ptr(x, VEC) && wide_ptr(scale, 4) &&
                   wide_ptr(wide, VEC) && wide_ptr(w, 4) && wide_ptr(dout, VEC) && wide_ptr(dwide, VEC) && wide_ptr(dx, VEC) &&
                   wide_ptr(dwide_out, VEC);
  cudaError_t e = cudaSuccess;
  auto rows = [&](auto nv, auto v) {
    return norm_backward_rows<M, TX, TR, decltype(v)::value, decltype(nv)::value>(
        x, scale, wide, w, eps, dout, dwide, dx, dwide_out, pw, ps, d, parts, e, st);
  };
  // 8 or 16 channels a thread.  The residual norm's two vectors of sums fill the registers at 8 (65536 x 768, bf16
  // with an fp32 stream: 195 us, at 16 330); the gated norm's one leaves room for 16, and half the reductions a row
  // (4096 x 5120: 71 us, at 8 92), unless more lanes are left idle than at 8 (43690 x 768: 136 us, at 8 96).  Rows
  // too long for 8 take 16 in any case.
  const int64_t W = d.D / d.G;
  auto idle = [&](int n) {
    const Split p = split_unit((W + VEC - 1) / VEC, n / VEC, n / VEC, [](int) { return kRowThreads; });
    return p.tpr == 0 ? INT64_MAX : p.tpr * n - W;
  };
  const bool more = M == kResidual ? idle(8) == INT64_MAX : idle(16) <= idle(8);
  bool done;
  if (vec)
    done = more ? rows(std::integral_constant<int, 16 / VEC>{}, std::integral_constant<int, VEC>{})
                : rows(std::integral_constant<int, 8 / VEC>{}, std::integral_constant<int, VEC>{});
  else
    done = rows(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  if (!done)
    e = launch(k_norm_backward<M, TX, TR>, dim3((unsigned)parts), kThreads, 0, st, false, x, scale, wide, w, eps, dout, dwide,
               dx, dwide_out, pw, ps, d);
  if (e != cudaSuccess || (dw == nullptr && ds == nullptr)) return e;
  return launch_row_sums(pw, ps, dw, ds, d.D, parts, st);
}

}  // namespace

cudaError_t launch_row_sums(const float *p0, const float *p1, float *o0, float *o1, int64_t D, int64_t n,
                            cudaStream_t st) {
  return launch_dependent(k_row_sums, dim3((unsigned)((D + 31) / 32), o1 != nullptr ? 2 : 1), 1024, 0, st, p0, p1, o0,
                          o1, D, n);
}

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
