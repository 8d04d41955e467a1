// glr.cu -- the gated linear recurrence, one state value per channel:
//
//   L_t = A sigmoid(r_t),  a_t = exp(L_t),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t
//
// over whole sequences, for one token, and its gradients.
#include <algorithm>

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

// a = exp(L) for L <= 0, in one register: a itself where L < -0.5, else u = a - 1 (<= 0).  Near
// zero u comes from its Taylor series (the first term left out is below 0.5^8 / 9! = 1e-8 of
// the sum), so that a = 1 + u and 1 - a^2 = -u (2 + u) keep full relative precision for decays
// close to 1; an exp(L) rounded near 1 and subtracted would not, and its error would be
// carried through every step of a long memory.  Further away the exponential itself keeps a
// small a precise (the floor of 1e-37 keeps it positive, hence recognisable).
__device__ __forceinline__ float pack_decay(float L) {
  float p = 1.f / 40320.f;
  p = fmaf(p, L, 1.f / 5040.f);
  p = fmaf(p, L, 1.f / 720.f);
  p = fmaf(p, L, 1.f / 120.f);
  p = fmaf(p, L, 1.f / 24.f);
  p = fmaf(p, L, 1.f / 6.f);
  p = fmaf(p, L, 0.5f);
  p = fmaf(p, L, 1.f);
  return L < -0.5f ? fmaxf(ex2(L * kLog2e), 1e-37f) : p * L;
}
__device__ __forceinline__ float packed_a(float w) { return w > 0.f ? w : 1.f + w; }
__device__ __forceinline__ float packed_rest(float w) {  // 1 - a^2
  const float u = w > 0.f ? w - 1.f : w;
  return -u * (2.f + u);
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

// One step back: c (in: c_{t+1}, out: c_t = a_t g_t), the gradients of x, r and i, and dA's term.
// dx = g beta si; di = dx x (1 - si); dL = g (a h_{t-1} - a^2 / beta si x); dr = dL L (1 - sr).
// Where beta is 0 (a = 1) its slope's term is taken as 0.
__device__ __forceinline__ void slopes(float A, float w, float zr, float r, float i, float x, float before, float dh,
                                       float &c, float &dx, float &dr, float &di, float &dA) {
  const float a = packed_a(w), rest = packed_rest(w);
  const float inv = rest > 1e-37f ? rsqrt_approx(rest) : 0.f, beta = rest * inv;
  const float zi = sigmoid_small(i), six = pick(i, zi), sr = pick(r, zr);
  const float g = dh + c;
  c = a * g;
  dx = g * beta * six;
  di = dx * x * pick(-i, zi);
  const float dL = c * (before - a * inv * six * x);
  dr = dL * (A * sr) * pick(-r, zr);
  dA = fmaf(dL, sr, dA);
}

// One step: the decay a and the input term b = sqrt(1 - a^2) sigmoid(i) x.
__device__ __forceinline__ void gate(float x, float r, float i, float A, float &a, float &b) {
  const float w = pack_decay(A * pick(r, sigmoid_small(r)));
  a = packed_a(w);
  b = sqrt_approx(packed_rest(w)) * pick(i, sigmoid_small(i)) * x;
}

// The scans.  A CTA takes 64 channels (two a lane) of one batch row and walks the sequence in
// tiles of 64 tokens, 8 a warp.  Each warp copies its own tokens of the next tiles into
// shared memory (two stages) while it forms the gates of this one, keeps its 8 decays and
// input terms in registers, and publishes what they do to a state, h -> A h + H, as one
// float4 a lane.  After a barrier a warp applies the warps before it to the carried state and
// runs its 8 steps: every array is read and written once.  Where the channels alone leave
// the GPU idle, a cluster of up to 8 CTAs shares a sequence, a tile each in turn: the CTAs'
// own A h + H go to the ranks behind them through distributed shared memory.
constexpr int kW = 8;          // warps
constexpr int kT = 8;          // tokens a warp
constexpr int kTile = kW * kT;
constexpr int kCh = 64;        // channels a CTA
constexpr int kMaxRanks = 8;

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// CW bytes global -> shared, zeros when !valid (nothing is read then)
template <int CW>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool valid) {
  const int n = valid ? CW : 0;
  if constexpr (CW == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void commit_async() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_async() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's copy of rows t .. t + 7 (of those in [0, L)) of 64 channels from c0 on.  `base` is
// the batch row's first element.  CW: bytes a copy (16 or 4), or 0 for element loads.
template <typename T, int CW>
__device__ __forceinline__ void fetch(T *dst, const T *base, int64_t t, int64_t L, int64_t stride, int64_t c0,
                                      int64_t D, int lane) {
  if constexpr (CW == 0) {
#pragma unroll
    for (int q = 0; q < kT * kCh / 32; ++q) {
      const int row = q * 32 / kCh, c = q * 32 % kCh + lane;
      const int64_t tt = t + row;
      const bool valid = tt >= 0 && tt < L && c0 + c < D;
      dst[row * kCh + c] = valid ? base[tt * stride + c0 + c] : T(0.f);
    }
  } else {
    constexpr int E = CW / (int)sizeof(T), CPR = kCh / E, N = kT * CPR / 32;  // elements a copy, copies a row
    const uint32_t to = smem_addr(dst) + lane * CW;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const int row = CPR <= 32 ? q * (32 / CPR) + lane / CPR : q / (CPR / 32);
      const int c = (CPR <= 32 ? lane % CPR : q % (CPR / 32) * 32 + lane) * E;
      const int64_t tt = t + row;
      const bool valid = tt >= 0 && tt < L && c0 + c < D;
      copy_async<CW>(to + q * 32 * CW, valid ? base + tt * stride + c0 + c : base, valid);
    }
  }
}

__device__ __forceinline__ float2 pair(const float *p) { return *reinterpret_cast<const float2 *>(p); }
__device__ __forceinline__ float2 pair(const __nv_bfloat16 *p) {
  const uint32_t u = *reinterpret_cast<const uint32_t *>(p);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// Two neighbouring channels out; kPair: the address is aligned for both and both exist.
template <bool kPair, typename T>
__device__ __forceinline__ void store2(T *p, float u, float v, int n) {
  if constexpr (kPair) {
    if (n < 2) return;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2 *>(p) = make_float2(u, v);
    else
      *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(u, v);
  } else {
    if (n > 0) p[0] = from_f32<T>(u);
    if (n > 1) p[1] = from_f32<T>(v);
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// A barrier of the cluster: every write to distributed shared memory before it is seen after.
__device__ __forceinline__ void sync_ranks() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_rank(void *p, uint32_t rank, float4 v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// State updates h -> A h + H of two channels {A0, H0, A1, H1}: `second` after `first`.
__device__ __forceinline__ float4 then(float4 first, float4 second) {
  return make_float4(first.x * second.x, fmaf(second.x, first.y, second.y), first.z * second.z,
                     fmaf(second.z, first.w, second.w));
}
__device__ __forceinline__ float2 apply(float4 f, float2 h) {
  return make_float2(fmaf(f.x, h.x, f.y), fmaf(f.z, h.y, f.w));
}

// What the warps and ranks of a scan tell one another, by parity of the tile.
struct Links {
  float4 warp[2][kW][32];
  float4 rank[2][kMaxRanks][32];
  float4 carry[2][32];  // x, y: the state entering the tile
};

// The state entering this warp's tokens, given its own update `mine`; all ranks call it once a tile.
template <bool kCluster>
__device__ __forceinline__ float2 enter(Links &l, int par, int warp, int lane, int rank, int ranks, float4 mine) {
  l.warp[par][warp][lane] = mine;
  __syncthreads();
  float4 before = make_float4(1.f, 0.f, 1.f, 0.f);
  for (int w = 0; w < warp; ++w) before = then(before, l.warp[par][w][lane]);
  if constexpr (kCluster) {
    if (warp == kW - 1) {
      const float4 all = then(before, mine);
      for (int k = rank + 1; k < ranks; ++k) store_rank(&l.rank[par][rank][lane], k, all);
    }
    sync_ranks();
  }
  const float4 c = l.carry[par][lane];
  float2 h = make_float2(c.x, c.y);
  if constexpr (kCluster)
    for (int k = 0; k < rank; ++k) h = apply(l.rank[par][k][lane], h);
  return apply(before, h);
}
// The state after the tile's last token, from the last warp of the last rank, for the next tile (not
// after the last one: a rank may have left by then).
template <bool kCluster>
__device__ __forceinline__ void leave(Links &l, int par, int lane, int ranks, float2 h) {
  const float4 v = make_float4(h.x, h.y, 0.f, 0.f);
  if constexpr (kCluster)
    for (int k = 0; k < ranks; ++k) store_rank(&l.carry[par ^ 1][lane], k, v);
  else
    l.carry[par ^ 1][lane] = v;
}

template <typename T, int N>
struct ScanSmem {
  T in[kW][2][N][kT][kCh];
  Links links;
};

template <typename T, int CW, bool kCluster>
__global__ void __launch_bounds__(kW * 32, sizeof(T) == 2 ? 3 : 2)
    k_glr_prefill(const T *__restrict__ x, const T *__restrict__ r, const T *__restrict__ i,
                  const float *__restrict__ A, const float *init, T *__restrict__ h, float *final_state, GlrDims d,
                  int blocks) {
  extern __shared__ __align__(16) char raw[];
  ScanSmem<T, 3> &sm = *reinterpret_cast<ScanSmem<T, 3> *>(raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = kCluster ? cluster_rank() : 0, ranks = kCluster ? cluster_size() : 1;
  const int64_t blk = blockIdx.x / ranks, b = blk / blocks, c0 = blk % blocks * kCh, c = c0 + 2 * lane;
  const int n = (int)max((int64_t)0, min((int64_t)2, d.D - c));  // channels of this lane
  const float A0 = n > 0 ? A[c] : 0.f, A1 = n > 1 ? A[c + 1] : 0.f;
  const T *const in[3] = {x + b * d.L * d.row, r + b * d.L * d.row, i + b * d.L * d.row};
  const int64_t tiles = (d.L + kTile * ranks - 1) / (kTile * ranks);
  auto first = [&](int64_t tile) { return (tile * ranks + rank) * kTile + warp * kT; };
  auto load = [&](int64_t tile) {
    if (tile < tiles) {
#pragma unroll
      for (int k = 0; k < 3; ++k)
        fetch<T, CW>(&sm.in[warp][tile & 1][k][0][0], in[k], first(tile), d.L, d.row, c0, d.D, lane);
    }
    commit_async();
  };
  load(0);
  load(1);
  if (warp == 0)
    sm.links.carry[0][lane] = init != nullptr ? make_float4(n > 0 ? init[b * d.D + c] : 0.f,
                                                            n > 1 ? init[b * d.D + c + 1] : 0.f, 0.f, 0.f)
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (kCluster) sync_ranks();  // no rank writes to another that has not started
  float2 s = make_float2(0.f, 0.f);
  for (int64_t tile = 0; tile < tiles; ++tile) {
    const int par = tile & 1;
    const int64_t t = first(tile);
    wait_async<1>();
    __syncwarp();
    float2 a[kT], v[kT];
    float4 all = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
    for (int j = 0; j < kT; ++j) {
      const float2 xj = pair(&sm.in[warp][par][0][j][2 * lane]), rj = pair(&sm.in[warp][par][1][j][2 * lane]),
                   ij = pair(&sm.in[warp][par][2][j][2 * lane]);
      gate(xj.x, rj.x, ij.x, A0, a[j].x, v[j].x);
      gate(xj.y, rj.y, ij.y, A1, a[j].y, v[j].y);
      if (t + j >= d.L) a[j] = make_float2(1.f, 1.f), v[j] = make_float2(0.f, 0.f);
      all = then(all, make_float4(a[j].x, v[j].x, a[j].y, v[j].y));
    }
    __syncwarp();
    load(tile + 2);
    s = enter<kCluster>(sm.links, par, warp, lane, rank, ranks, all);
    T *out = h + (b * d.L + t) * d.D + c;
#pragma unroll
    for (int j = 0; j < kT; ++j) {
      s = make_float2(fmaf(a[j].x, s.x, v[j].x), fmaf(a[j].y, s.y, v[j].y));
      if (t + j < d.L) store2<CW == 16>(out + j * d.D, s.x, s.y, n);
    }
    if (warp == kW - 1 && rank == ranks - 1 && tile + 1 < tiles) leave<kCluster>(sm.links, par, lane, ranks, s);
  }
  if (warp == kW - 1 && rank == ranks - 1) store2<false>(final_state + b * d.D + c, s.x, s.y, n);
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

// The reverse scan: c_t = a_t g_t with g_t = dh_t + c_{t+1}, that is c_t = a_t c_{t+1} + a_t dh_t, over
// tiles from the sequence's end.  Of the gates only the decay is needed before the barrier; it is kept
// with sigmoid(r), and the rest is formed when g is known.  A tile is 5 inputs deep, which leaves two CTAs
// an SM for bf16 and one for fp32.
template <typename T, int CW, bool kCluster>
__global__ void __launch_bounds__(kW * 32, sizeof(T) == 2 ? 2 : 1)
    k_glr_backward(const T *__restrict__ x, const T *__restrict__ r, const T *__restrict__ i,
                   const float *__restrict__ A, const float *__restrict__ init, const T *__restrict__ h,
                   const T *__restrict__ dh, const float *dfinal, T *__restrict__ dx, T *__restrict__ dr,
                   T *__restrict__ di, float *dinit, float *__restrict__ part, GlrDims d, int blocks) {
  extern __shared__ __align__(16) char raw[];
  ScanSmem<T, 5> &sm = *reinterpret_cast<ScanSmem<T, 5> *>(raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = kCluster ? cluster_rank() : 0, ranks = kCluster ? cluster_size() : 1;
  const int64_t blk = blockIdx.x / ranks, b = blk / blocks, c0 = blk % blocks * kCh, c = c0 + 2 * lane;
  const int n = (int)max((int64_t)0, min((int64_t)2, d.D - c));
  const float A0 = n > 0 ? A[c] : 0.f, A1 = n > 1 ? A[c + 1] : 0.f;
  const int64_t tiles = (d.L + kTile * ranks - 1) / (kTile * ranks);
  // the first of a warp's tokens, t .. t + 7; those below 0 lie before the sequence
  auto first = [&](int64_t tile) { return d.L - ((tile * ranks + rank) * kTile + warp * kT) - kT; };
  auto load = [&](int64_t tile) {
    if (tile < tiles) {
      const int64_t t = first(tile), at = b * d.L * d.row, o = b * d.L * d.D;
      auto &in = sm.in[warp][tile & 1];
      fetch<T, CW>(&in[0][0][0], r + at, t, d.L, d.row, c0, d.D, lane);
      fetch<T, CW>(&in[1][0][0], dh + o, t, d.L, d.D, c0, d.D, lane);
      fetch<T, CW>(&in[2][0][0], i + at, t, d.L, d.row, c0, d.D, lane);
      fetch<T, CW>(&in[3][0][0], x + at, t, d.L, d.row, c0, d.D, lane);
      fetch<T, CW>(&in[4][0][0], h + o, t - 1, d.L, d.D, c0, d.D, lane);  // h_{t-1}
    }
    commit_async();
  };
  load(0);
  load(1);
  if (warp == 0)
    sm.links.carry[0][lane] =
        dfinal != nullptr ? make_float4(n > 0 ? dfinal[b * d.D + c] : 0.f, n > 1 ? dfinal[b * d.D + c + 1] : 0.f, 0.f, 0.f)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (kCluster) sync_ranks();  // no rank writes to another that has not started
  float2 s = make_float2(0.f, 0.f), dA = make_float2(0.f, 0.f);
  for (int64_t tile = 0; tile < tiles; ++tile) {
    const int par = tile & 1;
    const int64_t t = first(tile);
    wait_async<1>();
    __syncwarp();
    auto &in = sm.in[warp][par];
    float2 code[kT], zr[kT];
    float4 all = make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
    for (int j = kT - 1; j >= 0; --j) {
      const float2 rj = pair(&in[0][j][2 * lane]), gj = pair(&in[1][j][2 * lane]);
      zr[j] = make_float2(sigmoid_small(rj.x), sigmoid_small(rj.y));
      code[j] = t + j >= 0 ? make_float2(pack_decay(A0 * pick(rj.x, zr[j].x)), pack_decay(A1 * pick(rj.y, zr[j].y)))
                           : make_float2(0.f, 0.f);
      const float a0 = packed_a(code[j].x), a1 = packed_a(code[j].y);
      all = then(all, make_float4(a0, a0 * gj.x, a1, a1 * gj.y));
    }
    s = enter<kCluster>(sm.links, par, warp, lane, rank, ranks, all);
#pragma unroll
    for (int j = kT - 1; j >= 0; --j) {
      const float2 rj = pair(&in[0][j][2 * lane]), gj = pair(&in[1][j][2 * lane]), ij = pair(&in[2][j][2 * lane]),
                   xj = pair(&in[3][j][2 * lane]);
      float2 hj = pair(&in[4][j][2 * lane]);
      if (t + j == 0 && init != nullptr)
        hj = make_float2(n > 0 ? init[b * d.D + c] : 0.f, n > 1 ? init[b * d.D + c + 1] : 0.f);
      float2 ox, oi, orr;
      slopes(A0, code[j].x, zr[j].x, rj.x, ij.x, xj.x, hj.x, gj.x, s.x, ox.x, orr.x, oi.x, dA.x);
      slopes(A1, code[j].y, zr[j].y, rj.y, ij.y, xj.y, hj.y, gj.y, s.y, ox.y, orr.y, oi.y, dA.y);
      if (t + j >= 0) {
        const int64_t to = (b * d.L + t + j) * d.grad + c;
        store2<CW == 16>(dx + to, ox.x, ox.y, n);
        store2<CW == 16>(dr + to, orr.x, orr.y, n);
        store2<CW == 16>(di + to, oi.x, oi.y, n);
      }
    }
    __syncwarp();
    load(tile + 2);
    if (warp == kW - 1 && rank == ranks - 1 && tile + 1 < tiles) leave<kCluster>(sm.links, par, lane, ranks, s);
  }
  if (dinit != nullptr && warp == kW - 1 && rank == ranks - 1) store2<false>(dinit + b * d.D + c, s.x, s.y, n);
  // dA over the CTA's warps, in order
  wait_async<0>();
  __syncthreads();
  float2 *sums = reinterpret_cast<float2 *>(raw);
  sums[warp * 32 + lane] = dA;
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < kW; ++w) dA = make_float2(dA.x + sums[w * 32 + lane].x, dA.y + sums[w * 32 + lane].y);
    store2<false>(part + (b * ranks + rank) * d.D + c, dA.x, dA.y, n);
  }
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

bool wide(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// CTAs that share a sequence: as many as the GPU holds at once (`resident` an SM) and the
// sequence has tiles for.
int pick_ranks(int64_t ctas, int64_t L, int resident) {
  const int64_t room = (int64_t)148 * resident / ctas, tiles = (L + kTile - 1) / kTile;
  return (int)std::max<int64_t>(1, std::min<int64_t>({room, tiles, kMaxRanks}));
}

template <typename... P, typename... V>
cudaError_t launch_ranks(void (*f)(P...), int64_t ctas, int ranks, size_t smem, cudaStream_t st, V... v) {
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(ctas * ranks));
  cfg.blockDim = dim3(kW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim = {(unsigned)ranks, 1, 1};
  cfg.attrs = &at;
  cfg.numAttrs = ranks > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, f, v...);
}

template <typename T>
cudaError_t launch_glr_prefill(const T *x, const T *r, const T *i, const float *A, const float *init, T *h,
                               float *final_state, const GlrDims &d, cudaStream_t st) {
  const int64_t blocks = (d.D + kCh - 1) / kCh, ctas = blocks * d.b;
  constexpr int E = 16 / sizeof(T);
  const bool w16 = wide(x) && wide(r) && wide(i) && wide(h) && d.D % E == 0 && d.row % E == 0;
  const int ranks = pick_ranks(ctas, d.L, sizeof(T) == 2 ? 3 : 1);
  auto run = [&](auto *one, auto *many) {
    return launch_ranks(ranks > 1 ? many : one, ctas, ranks, sizeof(ScanSmem<T, 3>), st, x, r, i, A, init, h,
                        final_state, d, (int)blocks);
  };
  if (w16) return run(k_glr_prefill<T, 16, false>, k_glr_prefill<T, 16, true>);
  constexpr int CW = sizeof(T) == 4 ? 4 : 0;
  return run(k_glr_prefill<T, CW, false>, k_glr_prefill<T, CW, true>);
}

template <typename T>
cudaError_t launch_glr_decode_step(float *state, const T *x, const T *r, const T *i, const float *A, T *h,
                                   const GlrDims &d, cudaStream_t st) {
  const int64_t blocks = (d.D + 127) / 128;
  k_glr_decode<T><<<(unsigned)(blocks * d.b), 128, 0, st>>>(state, x, r, i, A, h, d, (int)blocks);
  return cudaGetLastError();
}

size_t glr_backward_floats(const GlrDims &d) { return (size_t)d.b * kMaxRanks * d.D; }

template <typename T>
cudaError_t launch_glr_backward(const T *x, const T *r, const T *i, const float *A, const float *init, const T *h,
                                const T *dh, const float *dfinal, T *dx, T *dr, T *di, float *dA, float *dinit,
                                float *part, const GlrDims &d, cudaStream_t st) {
  const int64_t blocks = (d.D + kCh - 1) / kCh, ctas = blocks * d.b;
  constexpr int E = 16 / sizeof(T);
  const bool w16 = wide(x) && wide(r) && wide(i) && wide(h) && wide(dh) && wide(dx) && wide(dr) && wide(di) &&
                   d.D % E == 0 && d.row % E == 0 && d.grad % E == 0;
  const int ranks = pick_ranks(ctas, d.L, sizeof(T) == 2 ? 2 : 1);
  auto run = [&](auto *one, auto *many) {
    return launch_ranks(ranks > 1 ? many : one, ctas, ranks, sizeof(ScanSmem<T, 5>), st, x, r, i, A, init, h, dh,
                        dfinal, dx, dr, di, dinit, part, d, (int)blocks);
  };
  constexpr int CW = sizeof(T) == 4 ? 4 : 0;
  cudaError_t e = w16 ? run(k_glr_backward<T, 16, false>, k_glr_backward<T, 16, true>)
                      : run(k_glr_backward<T, CW, false>, k_glr_backward<T, CW, true>);
  if (e != cudaSuccess) return e;
  k_glr_sum<<<(unsigned)((d.D + 127) / 128), 128, 0, st>>>(part, dA, d.D, d.b * ranks);
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
