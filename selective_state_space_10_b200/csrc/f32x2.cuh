// f32x2.cuh -- fp32 arithmetic on two values an instruction, and the approximate special functions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {

// Two neighbouring channels.  Kernels that are as close to the issue limit as to the memory's compute on these.
struct f2 {
  unsigned long long v;
};
__device__ __forceinline__ f2 mk(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ f2 both(float x) { return mk(x, x); }
__device__ __forceinline__ float2 split(f2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ f2 operator*(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 operator+(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

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
__device__ __forceinline__ float rsqrt_approx(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ f2 ex2(f2 v) {
  const float2 s = split(v);
  return mk(ex2(s.x), ex2(s.y));
}
__device__ __forceinline__ f2 rcp(f2 v) {
  const float2 s = split(v);
  return mk(rcp(s.x), rcp(s.y));
}
__device__ __forceinline__ f2 rsqrt_approx(f2 v) {
  const float2 s = split(v);
  return mk(rsqrt_approx(s.x), rsqrt_approx(s.y));
}

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + exp(-v)); exp may overflow, to a sigmoid of 0
__device__ __forceinline__ f2 sigmoid(f2 v) { return rcp(ex2(v * both(-kLog2e)) + both(1.f)); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// A bf16 pair in a word, and back (rounded to nearest even).
__device__ __forceinline__ f2 from_bf16x2(uint32_t u) {
  return mk(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t to_bf16x2(f2 f) {
  const float2 s = split(f);
  const __nv_bfloat162 b = __floats2bfloat162_rn(s.x, s.y);
  return *reinterpret_cast<const uint32_t *>(&b);
}

}  // namespace ssd
