// glr.cu -- the gated linear recurrence, one state value per channel:
//
//   L_t = A sigmoid(r_t),  a_t = exp(L_t),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t
//
// over whole sequences, for one token, and its gradients.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "per_device.h"
#include "sm100.cuh"

namespace ssd {

namespace {

// maximum and minimum that keep a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
constexpr float kTiny = 1.2e-38f;  // keeps a root's argument positive where 1 - a^2 is 0

// exp(-v), with overflow to infinity; exp_neg_finite stops at 2^126, so that e / (1 + e) stays 1
__device__ __forceinline__ f2 exp_neg(f2 v) { return ex2(v * both(-kLog2e)); }
__device__ __forceinline__ f2 exp_neg_finite(f2 v) {
  const float2 s = split(v * both(-kLog2e));
  return mk(ex2(min_nan(s.x, 126.f)), ex2(min_nan(s.y, 126.f)));
}

// a = exp(L) and v = 1 - a for L <= 0, both to full relative precision: L = n ln 2 + f with |f| <= ln 2 / 2,
// p = 1 - exp(f) by a polynomial (fitted with relative weights, with 1 and 1/2 kept; 1.8e-8 off at most, below half a
// step of fp32), a = 2^n (1 - p), v = (1 - 2^n) + 2^n p.  1 - a^2 = v (1 + a) then loses nothing for decays close
// to 1; an exp(L) rounded near 1 and subtracted would, and its error would be carried through every step of a
// long memory.  Nor is a formed as 1 - v, which would leave a small one the absolute precision of 1.  The exponential
// unit, which the gates already fill, is not used.
__device__ __forceinline__ void decay(f2 L, f2 &a, f2 &v) {
  const float2 s = split(L);
  L = mk(max_nan(s.x, -87.f), max_nan(s.y, -87.f));  // n >= -126
  const f2 t = fma2(L, both(kLog2e), both(12582912.f));  // 1.5 * 2^23: the integer lands in the low bits
  const f2 n = t + both(-12582912.f);
  const f2 f = fma2(n, both(-0.6931471805599453f), L);
  f2 p = both(-0.0013946497347205877f);
  p = fma2(p, f, both(-0.00836661085486412f));
  p = fma2(p, f, both(-0.04166628047823906f));
  p = fma2(p, f, both(-0.1666654348373413f));
  p = fma2(p, f, both(-0.5f));
  p = fma2(p, f, both(-1.f)) * f;  // 1 - exp(f)
  const float2 i = split(t);
  const f2 two_n = mk(__int_as_float((__float_as_int(i.x) << 23) + 0x3f800000),
                      __int_as_float((__float_as_int(i.y) << 23) + 0x3f800000));
  v = fma2(two_n, p, fma2(two_n, both(-1.f), both(1.f)));
  a = two_n * fma2(p, both(-1.f), both(1.f));
}

// One step: the decay a and the input term b = sqrt(1 - a^2) sigmoid(i) x, with rest = 1 - a^2 and o = 1 + exp(-i) as
// x rest / sqrt(rest o^2): one root in place of a root and a reciprocal.  kTiny leaves b exactly 0 where a is 1 or o
// infinite, and changes nothing from rest = 2e-31 on.  Where the root's argument overflows (i below -44) its sum in `args`
// is no longer finite, and b is 0: right for a shut gate, but a nearly shut one has to take gate_wide.
__device__ __forceinline__ void gate(f2 x, f2 r, f2 i, f2 A, f2 &a, f2 &b, f2 &args) {
  f2 v;
  decay(A * rcp(exp_neg(r) + both(1.f)), a, v);
  const f2 rest = fma2(v, a, v), o = exp_neg(i) + both(1.f), arg = o * o * (rest + both(kTiny));
  b = x * (rest * rsqrt_approx(arg));
  args = args + arg;
}
// The same for every i: a sigmoid down to the end of the normal range.  Its fifth special function for every token would
// take the 2.7B-shaped bf16 prefill to 50.3 us; the sum of the arguments, and this where it is needed, 48.1 us.
__device__ __forceinline__ void gate_wide(f2 x, f2 r, f2 i, f2 A, f2 &a, f2 &b) {
  f2 v;
  decay(A * rcp(exp_neg(r) + both(1.f)), a, v);
  const f2 rest = fma2(v, a, v);
  b = x * rcp(exp_neg(i) + both(1.f)) * (rest * rsqrt_approx(rest + both(kTiny)));
}
__device__ __forceinline__ bool finite(f2 args) {  // a sum of terms that are not negative
  const float2 s = split(args);
  return s.x + s.y < __int_as_float(0x7f800000);
}

// One step back: c (in: c_{t+1}, out: c_t = a_t g_t), the gradients of x, r and i, and dA's term.
// dx = g beta si; di = dx x (1 - si); dL = g (a h_{t-1} - a^2 / beta si x); dr = dL L (1 - sr).
// Where beta is 0 (a = 1) its slope's term is taken as 0.
__device__ __forceinline__ void slopes(f2 A, f2 a, f2 v, f2 r, f2 i, f2 x, f2 before, f2 dh, f2 &c, f2 &dx, f2 &dr,
                                       f2 &di, f2 &dA) {
  const f2 rest = v * (a + both(1.f));
  const float2 q = split(rest);
  const f2 inv = mk(q.x > kTiny ? rsqrt_approx(q.x) : 0.f, q.y > kTiny ? rsqrt_approx(q.y) : 0.f);
  const f2 er = exp_neg_finite(r), ei = exp_neg_finite(i);
  const f2 sr = rcp(er + both(1.f)), si = rcp(ei + both(1.f)), six = si * x;
  const f2 g = dh + c, gb = g * (rest * inv);
  c = a * g;
  dx = gb * si;
  di = gb * six * (ei * si);
  const f2 dL = c * fma2(a * inv * six, both(-1.f), before), ds = dL * sr;
  dr = ds * A * (er * sr);
  dA = dA + ds;
}

__device__ __forceinline__ f2 load2(const float *p) {
  f2 r;
  r.v = *reinterpret_cast<const unsigned long long *>(p);
  return r;
}
__device__ __forceinline__ f2 load2(const __nv_bfloat16 *p) {
  return from_bf16x2(*reinterpret_cast<const uint32_t *>(p));
}
// The first n (0 .. 2) of two neighbouring channels, one by one.
template <typename T>
__device__ __forceinline__ f2 load_n(const T *p, int n) {
  return mk(n > 0 ? to_f32(p[0]) : 0.f, n > 1 ? to_f32(p[1]) : 0.f);
}
// Out; kPair: the address is aligned for both, and n is 0 or 2.
template <bool kPair, typename T>
__device__ __forceinline__ void store2(T *p, f2 f, int n) {
  const float2 s = split(f);
  if constexpr (kPair) {
    if (n == 0) return;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2 *>(p) = s;
    else
      *reinterpret_cast<uint32_t *>(p) = to_bf16x2(f);
  } else {
    if (n > 0) p[0] = from_f32<T>(s.x);
    if (n > 1) p[1] = from_f32<T>(s.y);
  }
}

// The scans.  A CTA takes 64 channels (two a lane) of one batch row and walks the sequence in
// tiles, kT tokens a warp.  Each warp copies its own tokens of the next tiles into shared memory
// (two stages) while it forms the gates of this one, keeps its decays and input terms in
// registers, and publishes what they do to a state, h -> A h + H, as one 16-byte word a lane.
// After a barrier a warp applies the warps before it to the carried state and runs its steps:
// every array is read and written once.  Where the channels alone leave the GPU idle, a cluster
// of CTAs shares a sequence, a tile each in turn: the CTAs' own A h + H go to the ranks behind
// them through distributed shared memory.
// Warps, tokens a warp and CTAs an SM of each scan.  Long runs of tokens amortise a tile's exchange, small CTAs keep the
// SMs evenly loaded (before the last steps; 2.7B-shaped bf16 prefill: 4 x 16 47.8 us, 4 x 12 54.0, 4 x 8 54.3, 2 x 16 57.2,
// 8 x 16 66.5 us; long-context bf16 gradient: 4 x 12 381 us, 4 x 8 408, 2 x 12 437, 4 x 4 490, 8 x 8 509 us).  fp32 tiles are
// twice the bytes; the prefill runs the same with any of these shapes, and the gradient's short runs leave room for four
// CTAs (b = 4, L = 4096, D = 5120: 4 x 4 442 us, 4 x 8 507 us; b = 1, L = 16384, D = 1536: 182 and 150 us).
template <typename T>
struct PrefillShape {
  static constexpr int W = 4, N = sizeof(T) == 2 ? 16 : 8, kResident = 3;
};
template <typename T>
struct BackwardShape {
  static constexpr int W = 4, N = sizeof(T) == 2 ? 12 : 4, kResident = sizeof(T) == 2 ? 3 : 4;
};
constexpr int kCh = 64;  // channels a CTA
constexpr int kMaxRanks = 16;
constexpr int64_t kMaxCtas = 148 * 4;  // of a launch whose CTAs share sequences

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
template <int CW>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void commit_async() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_async() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A lane's share of a warp's copies of kT token rows of 64 channels from c0 on.  CW: bytes a
// copy (16 or 4), or 0 for element loads.  The pointer follows the warp's rows from tile to
// tile; rows outside [lo, hi) and channels outside the array arrive as zeros.
template <typename T, int CW, int kT>
struct Rows {
  static constexpr int E = CW > 0 ? CW / (int)sizeof(T) : 1;  // elements a copy
  static constexpr int CPR = kCh / E;                         // copies a row
  static constexpr int N = kT * CPR / 32;                     // copies a lane
  const T *p;
  __device__ __forceinline__ static int row(int q, int lane) {
    return CPR <= 32 ? q * (32 / CPR) + lane / CPR : q / (CPR / 32);
  }
  __device__ __forceinline__ static int chan(int q, int lane) {
    return (CPR <= 32 ? lane % CPR : q % (CPR / 32) * 32 + lane) * E;
  }
  // t0: the warp's first token of the first tile (any integer: rows before the array are never read)
  __device__ __forceinline__ void start(const T *base, int64_t t0, int64_t stride, int64_t c0, int lane) {
    p = base + (t0 + row(0, lane)) * stride + c0 + chan(0, lane);
  }
  __device__ __forceinline__ const T *from(int q, int64_t stride) const {
    return p + (row(q, 0) - row(0, 0)) * stride + (chan(q, 0) - chan(0, 0));
  }
  // whole: every row and channel is there; array: where the others point instead (and nothing is read)
  __device__ __forceinline__ void fetch(T *dst, bool whole, int lo, int hi, int64_t stride, int64_t channels, int lane,
                                        const T *array) const {
    const uint32_t to = smem_addr(dst) + lane * E * (int)sizeof(T);
    if (CW == 16 && whole) {
#pragma unroll
      for (int q = 0; q < N; ++q) copy_async<16>(to + q * 32 * 16, from(q, stride));
      return;
    }
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const int j = row(q, lane);
      const bool valid = j >= lo && j < hi && chan(q, lane) < channels;
      if constexpr (CW == 0)
        dst[q * 32 + lane] = valid ? *from(q, stride) : T(0.f);
      else
        copy_async<CW>(to + q * 32 * CW, valid ? from(q, stride) : array, valid);
    }
  }
};

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
// The cluster's barrier; what was written to (distributed) shared memory before it is seen after.
__device__ __forceinline__ void sync_ranks() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void pause(uint64_t ns) {
  const uint64_t t0 = sm100::globaltimer_ns();
  while (sm100::globaltimer_ns() - t0 < ns) __nanosleep(10000);
}

// A state update h -> A h + H of a lane's two channels.
struct alignas(16) Link {
  f2 A, H;
};
__device__ __forceinline__ Link then(Link first, Link second) {
  return {first.A * second.A, fma2(second.A, first.H, second.H)};
}
// What the warps and ranks of a scan tell one another, by parity of the tile.
template <int kW>
struct Links {
  Link warp[2][kW][32];
  f2 carry[2][32];      // without a cluster: the state entering the tile
  uint64_t arrived[2];  // in one, mbarriers: the ranks' messages of a tile are here
  // behind it, in a cluster: Link rank[2][ranks][32]
};
__device__ __forceinline__ Link load_link(const Link &l) {
  const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(&l);
  return {{u.x}, {u.y}};
}

// The exchange of a tile: `publish` gives a warp's own update away, `collect` returns the state that enters its
// tokens, `leave` ends the tile with the state after them; every warp of every rank calls each once a tile.  In a
// cluster every warp keeps the state that enters the tile itself, from the updates of all ranks, so no tile waits for
// the steps of the one before; in a lone CTA its last warp hands it on.  The ranks' updates travel as st.async messages
// that count themselves in on the receiver's mbarrier: no warp waits for its own stores to drain, as it would at a cluster
// barrier a tile (2.7B-shaped bf16 prefill, 5 ranks: 47.8 us against 52.6 us).  Two slots are enough: a rank sends tile
// k + 2 after it has collected k + 1, which every rank published after all its warps had collected k.
// A wait gives up after kWaitLimit of global time.  What the lane forms from there on is NaN; at its CTA's next barrier
// the whole CTA is lost: it waits and sends no more.  So it reuses no slot that may still be read, and every other rank
// waits in vain at the next tile and is lost in turn: what is finite is right, and every later tile is NaN.
constexpr uint64_t kWaitLimit = 2000000000ull;  // ns
template <bool kCluster, int kW>
struct Exchange {
  Links<kW> &l;
  int warp, lane, rank, ranks;
  int par, phase;  // of the tile
  bool lost;       // a wait has expired: this lane's, or after a barrier any of the CTA
  Link before;     // the warps before this one
  f2 state;        // enters the tile
  uint64_t limit;  // of a wait

  // All threads of all ranks, once: `enters` the first tile.
  __device__ __forceinline__ Exchange(Links<kW> &links, int warp, int lane, int rank, int ranks, f2 enters,
                                      uint64_t limit = kWaitLimit)
      : l(links), warp(warp), lane(lane), rank(rank), ranks(ranks), par(0), phase(0), lost(false), state(enters),
        limit(limit) {
    if (!kCluster && warp == 0) l.carry[0][lane] = enters;
    if constexpr (kCluster) {
      if (threadIdx.x == 0) {
        sm100::mbar_init(&l.arrived[0], 1);
        sm100::mbar_init(&l.arrived[1], 1);
        sm100::mbar_fence_init();
      }
      sync_ranks();
    }
  }
  __device__ __forceinline__ Link *from_rank(int k) const {
    return reinterpret_cast<Link *>(&l + 1) + (par * ranks + k) * 32 + lane;
  }
  // One lane's 16 bytes of this rank's message of 512 to rank k.
  __device__ __forceinline__ void send(int k, Link v) const {
    uint32_t a, b;
    const float2 A = split(v.A), H = split(v.H);
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(from_rank(rank))), "r"(k));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_addr(&l.arrived[par])), "r"(k));
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
                 "f"(A.x), "f"(A.y), "f"(H.x), "f"(H.y), "r"(b)
                 : "memory");
  }
  __device__ __forceinline__ bool wait() const {
    const uint32_t bar = smem_addr(&l.arrived[par]);
    uint64_t t0 = 0;
    while (true) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(bar), "r"(phase), "r"(20000u)
          : "memory");
      if (ok) return true;
      const uint64_t t = sm100::globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > limit) return false;
    }
  }
  __device__ __forceinline__ void publish(Link mine) {
    l.warp[par][warp][lane] = mine;
    if constexpr (kCluster)
      lost = __syncthreads_or(lost);
    else
      __syncthreads();
    before = {both(1.f), both(0.f)};
    for (int w = 0; w < warp; ++w) before = then(before, load_link(l.warp[par][w][lane]));
    if constexpr (kCluster) {
      if (warp == kW - 1 && !lost) {
        const Link all = then(before, mine);
        if (lane == 0) sm100::mbar_arrive_expect_tx(&l.arrived[par], 512u * ranks);
        for (int k = 0; k < ranks; ++k) send(k, all);
      }
    }
  }
  __device__ __forceinline__ f2 collect() {
    f2 h = kCluster ? state : l.carry[par][lane];  // enters this CTA's tokens
    if constexpr (kCluster) {
      if (!lost) lost = !wait();
#pragma unroll 4
      for (int k = 0; k < ranks; ++k) {
        const Link f = load_link(*from_rank(k));
        if (k == rank) h = state;
        state = fma2(f.A, state, f.H);
      }
      if (lost) h = state = both(__int_as_float(0x7fffffff));
    }
    return fma2(before.A, h, before.H);
  }
  __device__ __forceinline__ void leave(f2 h) {
    if (!kCluster && warp == kW - 1) l.carry[par ^ 1][lane] = h;
    phase ^= par;
    par ^= 1;
  }
  __device__ __forceinline__ bool last() const { return warp == kW - 1 && rank == ranks - 1; }
  // No rank leaves while another may still write to it: each has collected all that was sent to it, but for a lost one,
  // which gives the last messages, all sent before the barrier, a millisecond to land.
  __device__ __forceinline__ void finish() {
    if constexpr (kCluster) {
      lost = __syncthreads_or(lost);
      sync_ranks();
      if (lost) pause(1000000);
    }
  }
};

template <typename T, int N, int kW, int kT>
struct ScanSmem {
  T in[kW][2][N][kT][kCh];
  Links<kW> links;  // the last member: the ranks' updates follow
};
template <typename T, int N, int kW, int kT>
size_t scan_smem(int ranks) {
  return sizeof(ScanSmem<T, N, kW, kT>) + (ranks > 1 ? 2 * ranks * 32 * sizeof(Link) : 0);
}

// A CTA's place in the grid.
struct Place {
  int warp, lane, rank, ranks, n;  // n: channels of this lane
  bool whole;                      // all 64 channels are there
  int64_t b, c0, c;
};
template <bool kCluster>
__device__ __forceinline__ Place place(int64_t D, int blocks) {
  Place p;
  p.warp = threadIdx.x / 32;
  p.lane = threadIdx.x % 32;
  p.rank = kCluster ? cluster_rank() : 0;
  p.ranks = kCluster ? cluster_size() : 1;
  const unsigned blk = blockIdx.x / p.ranks;
  p.b = blk / blocks;
  p.c0 = (int64_t)(blk % blocks) * kCh;
  p.c = p.c0 + 2 * p.lane;
  p.n = (int)max((int64_t)0, min((int64_t)2, D - p.c));
  p.whole = D - p.c0 >= kCh;
  return p;
}

// The input terms of a warp's tokens where a gate of the lane's may be nearly shut (its sum of arguments is not finite).
// Below kShut, where masks put a gate, the term is 0 already; up to kNearlyShut the terms take gate_wide, in a loop of one
// token at a time that leaves each term in the lane's own words of the tile and so takes no registers beside the decays.
// 2.7B-shaped bf16 prefill with one gate in 20 masked 50.8 us, all masked 51.8 us, all at -60 90 us.
constexpr float kShut = -87.4f, kNearlyShut = -44.f;  // 1 + exp(-i) is 2^126, its square 2^127
template <typename T, int kT>
__device__ __forceinline__ void shut_terms(T (&in)[3][kT][kCh], int lane, f2 A, f2 (&b)[kT]) {
  bool nearly = false;
#pragma unroll 4
  for (int j = 0; j < kT; ++j) {
    const float2 i = split(load2(&in[2][j][2 * lane]));
    nearly = nearly || (i.x >= kShut && i.x <= kNearlyShut) || (i.y >= kShut && i.y <= kNearlyShut);
  }
  if (!nearly) return;
#pragma unroll 1
  for (int j = 0; j < kT; ++j) {
    T *x = &in[0][j][2 * lane], *i = &in[2][j][2 * lane];
    f2 a, term;
    gate_wide(load2(x), load2(&in[1][j][2 * lane]), load2(i), A, a, term);
    const float2 s = split(term);
    *reinterpret_cast<float *>(x) = s.x;
    *reinterpret_cast<float *>(i) = s.y;
  }
#pragma unroll
  for (int j = 0; j < kT; ++j)
    b[j] = mk(*reinterpret_cast<const float *>(&in[0][j][2 * lane]), *reinterpret_cast<const float *>(&in[2][j][2 * lane]));
}

// The forward scan.  2.7B-shaped bf16 layer (b = 1, L = 4096, D = 5120): 48.1 us a call for 168 MB, 3.5 TB/s, 53 % of the
// measured copy bandwidth; fp32 57.2 us, 5.9 TB/s.  The bf16 scan has twice the elements a byte: 37 warp instructions and
// 4 special functions for each, issue slots 53 % and special-function units 46 % busy with the 10 warps an SM that 166
// registers leave; what remains is their latency, and that a tile is serial within its CTA: gates, barrier, messages,
// steps.  Forming the next tile's gates while a tile's exchange is under way (a second set of registers, 8 warps an SM)
// measured 64 us.
template <typename T, int CW, bool kCluster, int kW, int kT>
__global__ void __launch_bounds__(kW * 32, PrefillShape<T>::kResident)
    k_glr_prefill(const T *x, const T *r, const T *i, const float *A, const float *init, T *h, float *final_state,
                  GlrDims d, int blocks) {
  constexpr int kTile = kW * kT;
  extern __shared__ __align__(16) char raw[];
  ScanSmem<T, 3, kW, kT> &sm = *reinterpret_cast<ScanSmem<T, 3, kW, kT> *>(raw);
  sm100::grid_dep_launch();
  sm100::grid_dep_wait();
  const Place p = place<kCluster>(d.D, blocks);
  const f2 Ac = load_n(A + p.c, p.n);
  const int64_t step = (int64_t)kTile * p.ranks, tiles = (d.L + step - 1) / step;
  const int64_t t0 = p.rank * kTile + p.warp * kT;  // this warp's first token
  int64_t left = d.L - t0;                          // tokens from it to the end
  Rows<T, CW, kT> rows[3];
  rows[0].start(x + p.b * d.L * d.row, t0, d.row, p.c0, p.lane);
  rows[1].start(r + p.b * d.L * d.row, t0, d.row, p.c0, p.lane);
  rows[2].start(i + p.b * d.L * d.row, t0, d.row, p.c0, p.lane);
  auto load = [&](int stage, int64_t rest) {  // rest: tokens of the sequence from the first row on
    if (rest > 0) {
      const bool whole = p.whole && rest >= kT;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        rows[k].fetch(&sm.in[p.warp][stage][k][0][0], whole, 0, (int)min(rest, (int64_t)kT), d.row, d.D - p.c0, p.lane,
                      k == 0 ? x : k == 1 ? r : i);
        rows[k].p += step * d.row;
      }
    }
    commit_async();
  };
  // the gates of the tile in `stage`, of which the sequence has `rest` tokens
  auto gates = [&](int stage, int64_t rest, f2 (&a)[kT], f2 (&v)[kT]) {
    wait_async<1>();
    __syncwarp();
    auto &in = sm.in[p.warp][stage];
    auto at = [&](int k, int j) { return load2(&in[k][j][2 * p.lane]); };
    f2 args = both(0.f);
#pragma unroll
    for (int j = 0; j < kT; ++j) gate(at(0, j), at(1, j), at(2, j), Ac, a[j], v[j], args);
    if (rest > 0 && !finite(args)) shut_terms(in, p.lane, Ac, v);  // past the end there is whatever the tile held before
    if (rest < kT) {  // the sequence ends within these tokens: the rest leave the state as it is
#pragma unroll
      for (int j = 0; j < kT; ++j)
        if (j >= rest) a[j] = both(1.f), v[j] = both(0.f);
    }
    __syncwarp();
  };
  load(0, left);
  load(1, left - step);
  Exchange<kCluster, kW> ex(sm.links, p.warp, p.lane, p.rank, p.ranks,
                            init != nullptr ? load_n(init + p.b * d.D + p.c, p.n) : both(0.f));
  T *out = h + (p.b * d.L + t0) * d.D + p.c;
  f2 s = both(0.f);
  for (int64_t tile = 0; tile < tiles; ++tile, left -= step, out += step * d.D) {
    const int par = tile & 1;
    f2 a[kT], v[kT];
    gates(par, left, a, v);
    Link all = {a[0], v[0]};
#pragma unroll
    for (int j = 1; j < kT; ++j) all = then(all, {a[j], v[j]});
    ex.publish(all);
    load(par, left - 2 * step);  // while the ranks' messages travel
    s = ex.collect();
    if (left >= kT) {
#pragma unroll
      for (int j = 0; j < kT; ++j) {
        s = fma2(a[j], s, v[j]);
        store2<(CW >= 2 * (int)sizeof(T))>(out + j * d.D, s, p.n);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kT; ++j) {
        s = fma2(a[j], s, v[j]);
        if (j < left) store2<(CW >= 2 * (int)sizeof(T))>(out + j * d.D, s, p.n);
      }
    }
    ex.leave(s);
  }
  if (ex.last()) store2<false>(final_state + p.b * d.D + p.c, s, p.n);
  ex.finish();
}

// One token: 4 channels a thread in wide words (kWide), else two by elements.  256 x 5120 bf16 (21 MB read and written) in
// a graph of such steps: 3.7 us a step on the same arrays, which stay in L2, 4.7 us on eight sets in turn, 6.2 us by
// elements (5121 channels); 6.4 us alone and with the clocks that a profiler finds.  A call takes the host longer.
template <typename T, bool kWide>
__global__ void __launch_bounds__(128) k_glr_decode(float *state, const T *x, const T *r, const T *i,
                                                    const float *A, T *h, GlrDims d, int blocks) {
  constexpr int E = kWide ? 4 : 2;
  sm100::grid_dep_launch();
  sm100::grid_dep_wait();
  const int64_t b = blockIdx.x / blocks, c = ((int64_t)(blockIdx.x % blocks) * 128 + threadIdx.x) * E;
  const int64_t at = b * d.row + c, s = b * d.D + c;
  if constexpr (kWide) {
    if (c >= d.D) return;
    const float4 xv = load4(x + at), rv = load4(r + at), iv = load4(i + at), Av = load4(A + c), sv = load4(state + s);
    f2 a0, v0, a1, v1;
    gate_wide(mk(xv.x, xv.y), mk(rv.x, rv.y), mk(iv.x, iv.y), mk(Av.x, Av.y), a0, v0);
    gate_wide(mk(xv.z, xv.w), mk(rv.z, rv.w), mk(iv.z, iv.w), mk(Av.z, Av.w), a1, v1);
    v0 = fma2(a0, mk(sv.x, sv.y), v0);
    v1 = fma2(a1, mk(sv.z, sv.w), v1);
    const float2 lo = split(v0), hi = split(v1);
    const float4 next = make_float4(lo.x, lo.y, hi.x, hi.y);
    *reinterpret_cast<float4 *>(state + s) = next;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4 *>(h + s) = next;
    else
      *reinterpret_cast<uint2 *>(h + s) = make_uint2(to_bf16x2(v0), to_bf16x2(v1));
  } else {
    const int n = (int)max((int64_t)0, min((int64_t)2, d.D - c));
    f2 a, v;
    gate_wide(load_n(x + at, n), load_n(r + at, n), load_n(i + at, n), load_n(A + c, n), a, v);
    const f2 next = fma2(a, load_n(state + s, n), v);
    store2<false>(state + s, next, n);
    store2<false>(h + s, next, n);
  }
}

// The reverse scan: c_t = a_t g_t with g_t = dh_t + c_{t+1}, that is c_t = a_t c_{t+1} + a_t dh_t, over
// tiles from the sequence's end.  Of the gates only the decay is needed before the exchange; it is kept,
// and the rest is formed when g is known.  Long-context bf16 batch (b = 4, L = 16384, D = 1536): 380 to 392 us a call, by
// box, for 1.61 GB, 4.2 TB/s, 64 % of the measured copy bandwidth (370 us in a graph); issue slots 53 % busy, as in the
// forward scan.
template <typename T, int CW, bool kCluster, int kW, int kT>
__global__ void __launch_bounds__(kW * 32, BackwardShape<T>::kResident)
    k_glr_backward(const T *x, const T *r, const T *i, const float *A, const float *init, const T *h, const T *dh,
                   const float *dfinal, T *dx, T *dr, T *di, float *dinit, float *part, GlrDims d, int blocks) {
  constexpr int kTile = kW * kT;
  extern __shared__ __align__(16) char raw[];
  ScanSmem<T, 5, kW, kT> &sm = *reinterpret_cast<ScanSmem<T, 5, kW, kT> *>(raw);
  sm100::grid_dep_wait();
  const Place p = place<kCluster>(d.D, blocks);
  const f2 Ac = load_n(A + p.c, p.n);
  const int64_t step = (int64_t)kTile * p.ranks, tiles = (d.L + step - 1) / step;
  // this warp's tokens are t .. t + kT - 1; those below 0 lie before the sequence
  int64_t t = d.L - kT - (p.rank * kTile + p.warp * kT);
  Rows<T, CW, kT> rows[5];  // r, dh, i, x, h_{t-1}
  const int64_t at = p.b * d.L * d.row, o = p.b * d.L * d.D;
  rows[0].start(r + at, t, d.row, p.c0, p.lane);
  rows[1].start(dh + o, t, d.D, p.c0, p.lane);
  rows[2].start(i + at, t, d.row, p.c0, p.lane);
  rows[3].start(x + at, t, d.row, p.c0, p.lane);
  rows[4].start(h + o, t - 1, d.D, p.c0, p.lane);
  auto load = [&](int stage, int64_t t) {
    if (t > -kT) {
      const bool whole = p.whole && t > 0;
#pragma unroll
      for (int k = 0; k < 5; ++k) {
        const int64_t stride = k == 1 || k == 4 ? d.D : d.row;
        const int lo = (int)max((int64_t)0, (k == 4 ? 1 : 0) - t);
        rows[k].fetch(&sm.in[p.warp][stage][k][0][0], whole, lo, kT, stride, d.D - p.c0, p.lane,
                      k == 0 ? r : k == 1 ? dh : k == 2 ? i : k == 3 ? x : h);
        rows[k].p -= step * stride;
      }
    }
    commit_async();
  };
  load(0, t);
  load(1, t - step);
  Exchange<kCluster, kW> ex(sm.links, p.warp, p.lane, p.rank, p.ranks,
                            dfinal != nullptr ? load_n(dfinal + p.b * d.D + p.c, p.n) : both(0.f));
  int64_t to = (p.b * d.L + t) * d.grad + p.c;
  f2 s = both(0.f), dA = both(0.f);
  for (int64_t tile = 0; tile < tiles; ++tile, t -= step, to -= step * d.grad) {
    const int par = tile & 1;
    wait_async<1>();
    __syncwarp();
    const auto &in = sm.in[p.warp][par];
    f2 a[kT], v[kT];
#pragma unroll
    for (int j = kT - 1; j >= 0; --j)
      decay(Ac * rcp(exp_neg(load2(&in[0][j][2 * p.lane])) + both(1.f)), a[j], v[j]);
    if (t < 0) {  // tokens before the first leave c as it is
#pragma unroll
      for (int j = 0; j < kT; ++j)
        if (t + j < 0) a[j] = both(1.f), v[j] = both(0.f);
    }
    Link all = {both(1.f), both(0.f)};
    const bool any = t > -kT;  // a warp wholly before the sequence has fetched nothing
    if (any) {
#pragma unroll
      for (int j = kT - 1; j >= 0; --j) all = then(all, {a[j], a[j] * load2(&in[1][j][2 * p.lane])});
    }
    ex.publish(all);
    s = ex.collect();
#pragma unroll
    for (int j = kT - 1; j >= 0; --j) {
      if (!any) break;
      f2 before = load2(&in[4][j][2 * p.lane]);
      if (t + j == 0 && init != nullptr) before = load_n(init + p.b * d.D + p.c, p.n);
      f2 ox, orr, oi;
      slopes(Ac, a[j], v[j], load2(&in[0][j][2 * p.lane]), load2(&in[2][j][2 * p.lane]), load2(&in[3][j][2 * p.lane]),
             before, load2(&in[1][j][2 * p.lane]), s, ox, orr, oi, dA);
      if (t + j >= 0) {
        store2<(CW >= 2 * (int)sizeof(T))>(dx + to + j * d.grad, ox, p.n);
        store2<(CW >= 2 * (int)sizeof(T))>(dr + to + j * d.grad, orr, p.n);
        store2<(CW >= 2 * (int)sizeof(T))>(di + to + j * d.grad, oi, p.n);
      }
    }
    __syncwarp();
    load(par, t - 2 * step);
    ex.leave(s);
  }
  if (dinit != nullptr && ex.last()) store2<false>(dinit + p.b * d.D + p.c, s, p.n);
  // dA over the CTA's warps, in order
  wait_async<0>();
  __syncthreads();
  f2 *sums = reinterpret_cast<f2 *>(raw);
  sums[p.warp * 32 + p.lane] = dA;
  __syncthreads();
  if (p.warp == 0) {
    for (int w = 1; w < kW; ++w) dA = dA + sums[w * 32 + p.lane];
    store2<false>(part + (p.b * p.ranks + p.rank) * d.D + p.c, dA, p.n);
  }
  ex.finish();
}

// The exchange alone, with a limit and a rank that is late at one tile: every warp's update adds 1, and its state after
// each tile goes to out [tile][rank][warp][kCh].
__global__ void __launch_bounds__(4 * 32) k_glr_wait_selftest(float *out, int tiles, int late_rank, int late_tile,
                                                              uint64_t delay, uint64_t limit) {
  extern __shared__ __align__(16) char raw[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, rank = cluster_rank(), ranks = cluster_size();
  Exchange<true, 4> ex(*reinterpret_cast<Links<4> *>(raw), warp, lane, rank, ranks, both(1.f), limit);
  for (int tile = 0; tile < tiles; ++tile) {
    if (rank == late_rank && tile == late_tile) pause(delay);
    ex.publish({both(1.f), both(1.f)});
    const f2 s = ex.collect() + both(1.f);
    store2<true>(out + ((tile * ranks + rank) * 4 + warp) * kCh + 2 * lane, s, 2);
    ex.leave(s);
  }
  ex.finish();
}

// Bytes of a copy that every array's rows allow: 16, 4, or 0 (elements of 2).  2.7B-shaped bf16 prefill: 47 us with 16;
// two channels more, 62 us with 4; one more, 97 us by elements.
template <typename T>
int copy_width(std::initializer_list<const void *> arrays, std::initializer_list<int64_t> strides) {
  int width = 16;
  for (const void *p : arrays)
    while (width > 0 && reinterpret_cast<uintptr_t>(p) % width != 0) width = width == 16 ? 4 : 0;
  for (int64_t s : strides)
    while (width > 0 && s * (int64_t)sizeof(T) % width != 0) width = width == 16 ? 4 : 0;
  return width;
}
// run(std::integral_constant) for a width; elements of 4 bytes are aligned to 4.
template <typename T, typename F>
cudaError_t by_width(int width, F run) {
  if (width == 16) return run(std::integral_constant<int, 16>{});
  if constexpr (sizeof(T) == 2)
    if (width == 0) return run(std::integral_constant<int, 0>{});
  return run(std::integral_constant<int, 4>{});
}
bool wide(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// The launch of a scan kernel: `ranks` CTAs share a sequence and are a cluster.  The kernel's limits are set to the same
// values in every call: another thread's call with a size of its own may come between this and the launch.
template <typename T, int N, int kW, int kT, typename F>
cudaError_t set_up(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&at)[2], F *f, int64_t ctas, int ranks, cudaStream_t st) {
  cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3((unsigned)(ctas * ranks));
  cfg.blockDim = dim3(kW * 32);
  cfg.dynamicSmemBytes = scan_smem<T, N, kW, kT>(ranks);
  cfg.stream = st;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {(unsigned)ranks, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = ranks > 1 ? 2 : 1;
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)scan_smem<T, N, kW, kT>(kMaxRanks));
  if (e == cudaSuccess && ranks > 8) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

// How many CTAs share a sequence: the most, up to kMaxRanks, one a tile and kMaxCtas in all, whose clusters the GPU
// holds at once.
// What it holds depends on how clusters of a size fill its graphics clusters (2.7B-shaped prefill, 80 blocks of
// channels: 5 ranks 47.9 us, 4 56.0 us; 6 need a second wave, 59.6 us), so the runtime is asked, once for each kernel,
// size of a cluster and device.
template <typename T, int N, int kW, int kT, auto *many>
cudaError_t pick_ranks(int64_t ctas, int64_t L, int &ranks) {
  ranks = (int)std::min<int64_t>((L + kW * kT - 1) / (kW * kT), kMaxRanks);
  for (; ranks > 1; --ranks) {
    if (ctas * ranks > kMaxCtas) continue;
    int fit = 0;
    const cudaError_t e = clusters_held<many, kMaxRanks + 1>(ranks).get(fit, [&](int &clusters) {
      cudaLaunchConfig_t cfg;
      cudaLaunchAttribute at[2];
      const cudaError_t e = set_up<T, N, kW, kT>(cfg, at, many, 1, ranks, nullptr);
      return e != cudaSuccess ? e : cudaOccupancyMaxActiveClusters(&clusters, many, &cfg);
    });
    if (e != cudaSuccess) return e;
    if (ctas <= fit) break;
  }
  return cudaSuccess;
}

// `one`: the kernel of a lone CTA a sequence, `many`: of a cluster.  ranks: CTAs a sequence, as picked.
template <typename T, int N, int kW, int kT, auto *one, auto *many, typename... V>
cudaError_t launch_scan(int64_t ctas, int64_t L, int &ranks, cudaStream_t st, V... v) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute at[2];
  cudaError_t e = pick_ranks<T, N, kW, kT, many>(ctas, L, ranks);
  if (e != cudaSuccess) return e;
  auto *f = ranks > 1 ? many : one;
  e = set_up<T, N, kW, kT>(cfg, at, f, ctas, ranks, st);
  return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, f, v...);
}

}  // namespace

template <typename T>
cudaError_t launch_glr_prefill(const T *x, const T *r, const T *i, const float *A, const float *init, T *h,
                               float *final_state, const GlrDims &d, cudaStream_t st) {
  const int64_t blocks = (d.D + kCh - 1) / kCh, ctas = blocks * d.b;
  using Shape = PrefillShape<T>;
  constexpr int W = Shape::W, N = Shape::N;
  int ranks;
  auto run = [&](auto width) {
    constexpr int CW = decltype(width)::value;
    return launch_scan<T, 3, W, N, k_glr_prefill<T, CW, false, W, N>, k_glr_prefill<T, CW, true, W, N>>(
        ctas, d.L, ranks, st, x, r, i, A, init, h, final_state, d, (int)blocks);
  };
  return by_width<T>(copy_width<T>({x, r, i, h}, {d.D, d.row}), run);
}

template <typename T>
cudaError_t launch_glr_decode_step(float *state, const T *x, const T *r, const T *i, const float *A, T *h,
                                   const GlrDims &d, cudaStream_t st) {
  const bool w4 = wide(state) && wide(A) && wide(x) && wide(r) && wide(i) && wide(h) && d.D % 4 == 0 && d.row % 4 == 0;
  const int64_t per = 128 * (w4 ? 4 : 2), blocks = (d.D + per - 1) / per;
  auto *f = w4 ? k_glr_decode<T, true> : k_glr_decode<T, false>;
  return launch_dependent(f, dim3((unsigned)(blocks * d.b)), 128, 0, st, state, x, r, i, A, h, d, (int)blocks);
}

cudaError_t launch_glr_wait_selftest(float *out, int ranks, int tiles, int late_rank, int late_tile, uint64_t delay,
                                     uint64_t limit, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(4 * 32);
  cfg.dynamicSmemBytes = sizeof(Links<4>) + 2 * ranks * 32 * sizeof(Link);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim = {(unsigned)ranks, 1, 1};
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_glr_wait_selftest, out, tiles, late_rank, late_tile, delay, limit);
}

// A row of dim for each batch row and rank, of which there are at most kMaxCtas blocks of kCh where ranks > 1.
size_t glr_backward_floats(const GlrDims &d) { return (size_t)std::max(d.b * d.D, kMaxCtas * kCh); }

template <typename T>
cudaError_t launch_glr_backward(const T *x, const T *r, const T *i, const float *A, const float *init, const T *h,
                                const T *dh, const float *dfinal, T *dx, T *dr, T *di, float *dA, float *dinit,
                                float *part, const GlrDims &d, cudaStream_t st) {
  const int64_t blocks = (d.D + kCh - 1) / kCh, ctas = blocks * d.b;
  using Shape = BackwardShape<T>;
  constexpr int W = Shape::W, N = Shape::N;
  int ranks;
  auto run = [&](auto width) {
    constexpr int CW = decltype(width)::value;
    return launch_scan<T, 5, W, N, k_glr_backward<T, CW, false, W, N>, k_glr_backward<T, CW, true, W, N>>(
        ctas, d.L, ranks, st, x, r, i, A, init, h, dh, dfinal, dx, dr, di, dinit, part, d, (int)blocks);
  };
  const cudaError_t e = by_width<T>(copy_width<T>({x, r, i, h, dh, dx, dr, di}, {d.D, d.row, d.grad}), run);
  if (e != cudaSuccess) return e;
  return launch_row_sums(part, nullptr, dA, nullptr, d.D, d.b * ranks, st);
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
