// Gated linear recurrence per channel: h_t = a_t h_{t-1} + b_t x_t with a_t = exp(log_a_t) and
// b_t = 1, 1 - a_t or sqrt(1 - a_t^2); its gradients; and its single-token step.
//
// Forward and backward are one scan each.  The maps c -> A c + H of consecutive tokens compose
// to a map of the same form, so a run of tokens is known by two floats per channel.  A cluster
// of Z CTAs owns 32 channels of one batch entry and marches through time, Z tiles of 16 S tokens
// per step: lane = 2 channels, half a warp = S consecutive tokens (a segment), which it folds
// into one map; the CTA folds its 16 segments' maps and sends the result to every CTA of the
// cluster (st.async into their shared memory, which counts the bytes on an mbarrier there: a
// cluster barrier would also wait for the step's global stores).  From the Z maps each CTA has
// the carry into its tile and the carry into the next step, and the segments run their tokens
// from their carry, in registers.  Every input is read once and every output written once,
// nothing goes through global memory in between, and the folds have a fixed order, so results
// do not depend on timing.  The next tile's inputs are copied to shared memory (cp.async)
// while this one is worked on, and four small CTAs share an SM, so that one folds and waits
// while the others compute.
//
// What bounds them is issue and the exchange, not HBM: 75 instructions per token and pair of
// channels in the forward, 160 in the backward, and 512 CTAs that put four on some SMs and none on
// others.  With parts switched off, D 2048 bf16 with fp32 gates, b = sqrt(1 - a^2): the forward of T
// 16384 takes 68 us, 54 without the gates, 57.5 without the exchange between CTAs, 44.5 without
// both (HBM's time is 39.6); the backward of B4 T4096 120, 105, 110.5 and 94 (79.1).  That is 3.9 and
// 4.5 TB/s; the forward of B8 T2048, whose channel blocks have a CTA each, takes 57 us, 4.7 TB/s.
// Packed in 37 sequences with first states, 9001 tokens of 1000 channels, fp32: forward 33 us,
// backward 57.  Kept out of registers, the address of the sequences' bounds alone was worth 6%.
//
// Z is chosen so that batch entries x channel blocks x Z CTAs fill the GPU (launch_cluster).
// The backward is the same scan with time reversed.
//
// A sequence start is a reset: its map ignores the carry.  It is marked by A = -0.0 (a real A
// is never negative), not by A = 0, because 0 * inf would let an overflow of one sequence
// reach the next.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "ll_internal.cuh"
#include "tc_ptx.cuh"

namespace ll {

// bit 0: a step was given a slot that is out of range or given twice; bit 1: a wait for the
// cluster's maps ran out of time
__device__ unsigned int g_glr_error = 0;

namespace {

constexpr int kThreads = 256;
constexpr int kCh = 32;                      // channels of a CTA: two per lane
constexpr int kSegs = kThreads / (kCh / 2);  // segments of a tile
constexpr int kPerSm = 4;                    // CTAs per SM, shared memory permitting
constexpr int kMaxCluster = 16;

// ---------------------------------------------------------------- pairs of fp32

typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pack(float x, float y) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 both(float x) { return pack(x, x); }
__device__ __forceinline__ f32x2 to_pair(float2 v) { return pack(v.x, v.y); }

// ---------------------------------------------------------------- gates

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // relative error below 2^-22
  return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // relative error below 2^-22
  return y;
}

// a = exp(la) and m = 1 - a.  Gates live near a = 1, where 1 - a computed from a would lose the
// digits that la still has: for |la| <= 1/4 the Taylor sum of 1 - exp(la) (6 terms, its
// remainder is below 2^-24) gives m, and a from it to half a unit; beyond, exp itself is far
// enough from 1 (m off by 2^-20 at most).
__device__ __forceinline__ void gate_of(float2 la, f32x2* a, f32x2* m) {
  const f32x2 l = to_pair(la);
  f32x2 p = fma2(both(-1.f / 720.f), l, both(-1.f / 120.f));
  p = fma2(p, l, both(-1.f / 24.f));
  p = fma2(p, l, both(-1.f / 6.f));
  p = fma2(p, l, both(-0.5f));
  p = fma2(p, l, both(-1.f));
  const f32x2 m0 = mul2(p, l);
  const float2 s = unpack(mul2(l, both(1.44269504f)));
  const f32x2 e = pack(exp2_approx(s.x), exp2_approx(s.y));
  const float2 near_m = unpack(m0), near_a = unpack(fma2(m0, both(-1.f), both(1.f)));
  const float2 far_a = unpack(e), far_m = unpack(fma2(e, both(-1.f), both(1.f)));
  const bool nx = fabsf(la.x) <= 0.25f, ny = fabsf(la.y) <= 0.25f;
  *a = pack(nx ? near_a.x : far_a.x, ny ? near_a.y : far_a.y);
  *m = pack(nx ? near_m.x : far_m.x, ny ? near_m.y : far_m.y);
}

// b from m: 1 - a^2 = m (2 - m).  0 where a >= 1; a NaN stays one.
__device__ __forceinline__ float sqrt_clamped(float x) {
  float v;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(v) : "f"(x));
  return sqrt_approx(v);
}
template <int kScale>
__device__ __forceinline__ f32x2 scale_of(f32x2 m) {
  if (kScale == LL_GLR_ONE_MINUS) return m;
  if (kScale == LL_GLR_SQRT) {
    const float2 v = unpack(mul2(m, fma2(m, both(-1.f), both(2.f))));
    return pack(sqrt_clamped(v.x), sqrt_clamped(v.y));
  }
  return both(1.f);
}
// db / d log a.  The square root's is infinite at a = 1 and taken as 0 there.
template <int kScale>
__device__ __forceinline__ f32x2 scale_grad(f32x2 a, f32x2 b) {
  if (kScale == LL_GLR_ONE_MINUS) return mul2(a, both(-1.f));
  if (kScale == LL_GLR_SQRT) {
    const float2 q = unpack(mul2(a, mul2(a, both(-1.f)))), d = unpack(b);
    return pack(d.x > 0.f ? __fdividef(q.x, d.x) : 0.f, d.y > 0.f ? __fdividef(q.y, d.y) : 0.f);
  }
  return both(0.f);
}

// ---------------------------------------------------------------- element access

__device__ __forceinline__ float2 pair_of(const float* p) {
  return *reinterpret_cast<const float2*>(p);
}
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}
__device__ __forceinline__ void put_pair(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
__device__ __forceinline__ void put_pair(__nv_bfloat16* p, float2 v) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}

// How a pair of channels goes to global memory: both at once, one by one, or only the first.
enum { kPairs = 0, kSingles = 1, kFirst = 2 };
template <typename T>
__device__ __forceinline__ void store_pair(T* p, float2 v, int how) {
  if (how == kPairs) {
    put_pair(p, v);
  } else {
    p[0] = from_f32<T>(v.x);
    if (how == kSingles) p[1] = from_f32<T>(v.y);
  }
}
__device__ __forceinline__ float2 load_state(const float* p, int how) {
  return make_float2(p[0], how == kFirst ? 0.f : p[1]);
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// A tile in shared memory: 16 S tokens of 32 channels.  The two segments of a warp are read at
// once; bf16 rows are half a bank line, so odd segments have each pair of rows swapped.
template <typename T, int S>
struct Tile {
  T v[kSegs * S * kCh];
  static __device__ __forceinline__ int place(int row) {
    return sizeof(T) == 2 ? row ^ (row / S & 1) : row;
  }
  __device__ __forceinline__ T* at(int row, int ch) { return v + place(row) * kCh + ch; }
  __device__ __forceinline__ float2 pair(int seg, int s, int ch) const {
    const int odd = sizeof(T) == 2 ? seg & 1 : 0;
    return pair_of(v + seg * S * kCh + (s ^ odd) * kCh + ch);
  }
};

// Rows [lo, hi) of a tile of which `cols` channels exist, src addressing row 0.  bytes: the
// widest copy that pointers, strides and the number of channels allow (16, 4 or one element).
// What is not copied keeps its old contents, which no live lane uses.
template <typename T, int S>
__device__ __forceinline__ void fill(Tile<T, S>& dst, const T* src, int64_t stride, int lo, int hi,
                                     int cols, int bytes) {
  constexpr int rows = kSegs * S;
  if (bytes == 16) {
    constexpr int per = 16 / sizeof(T), chunks = kCh / per, pass = kThreads / chunks;
    const int r0 = threadIdx.x / chunks, c = (threadIdx.x % chunks) * per;
    if (lo == 0 && hi >= rows && cols == kCh && rows % pass == 0) {
      const T* p = src + r0 * stride + c;
#pragma unroll
      for (int r = 0; r < rows; r += pass) {
        cp_async16(dst.at(r0 + r, c), p);
        p += pass * stride;
      }
    } else {
#pragma unroll 1
      for (int r = r0; r < rows; r += pass) {
        if (r >= lo && r < hi && c < cols) cp_async16(dst.at(r, c), src + r * stride + c);
      }
    }
  } else if (bytes == 4) {
    constexpr int per = 4 / sizeof(T), chunks = kCh / per;
#pragma unroll 4
    for (int i = threadIdx.x; i < rows * chunks; i += kThreads) {
      const int r = i / chunks, c = (i % chunks) * per;
      if (r >= lo && r < hi && c < cols) tc::cp_async4(dst.at(r, c), src + r * stride + c, 4);
    }
  } else {
#pragma unroll 4
    for (int i = threadIdx.x; i < rows * kCh; i += kThreads) {
      const int r = i / kCh, c = i % kCh;
      if (r >= lo && r < hi && c < cols) *dst.at(r, c) = src[r * stride + c];
    }
  }
}

// ---------------------------------------------------------------- maps c -> A c + H

__device__ __forceinline__ float apply(float A, float H, float c) {
  return signbit(A) ? H : fmaf(A, c, H);
}
// A product of gates that are not 0 is not 0 here, but at least kLeast: an infinite carry stays
// infinite through gates however small, and becomes NaN through a gate of 0, as token by token.
// To a finite carry's part that makes a difference of at most 2^-149 of it.
constexpr float kLeast = 0x1p-149f;
// (A, H) after m, into m.
__device__ __forceinline__ void then(float2& m, float2 n) {
  m.y = apply(n.x, n.y, m.y);
  float t, p;  // t: the smaller factor, -0 where either is; p: a NaN stays one
  asm("min.f32 %0, %1, %2;" : "=f"(t) : "f"(n.x), "f"(m.x));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(p) : "f"(n.x * m.x), "f"(fminf(t, kLeast)));
  m.x = __uint_as_float(__float_as_uint(p) | (__float_as_uint(t) & 0x80000000u));
}
// Sets the products of the S gates of a segment, to[0].x and to[1].x, to kLeast where they came out as
// 0 and no gate is.  (Rare, and behind the store of the products: the backward's registers.)
template <int S>
__device__ __forceinline__ void keep_products(float2* to, f32x2 A, const f32x2 (&a)[S]) {
  const float2 p = unpack(A);
  const bool x = __float_as_uint(p.x) == 0, y = __float_as_uint(p.y) == 0;  // (-0 marks a reset)
  if (!x && !y) return;
  bool zx = false, zy = false;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const float2 g = unpack(a[s]);
    zx |= g.x == 0.f;
    zy |= g.y == 0.f;
  }
  if (x && !zx) to[0].x = kLeast;
  if (y && !zy) to[1].x = kLeast;
}

// ---------------------------------------------------------------- sequences

// The sequences of tokens [lo, lo + S): bit i of first / last: token lo + i begins / ends its
// sequence; of on: it belongs to one.  n0: the sequence that holds the first token that is on.
struct Span {
  uint32_t first, last, on;
  int n0;
};

// The tokens that need more than the recurrence, in either half of the warp: that are not there,
// or begin or end a sequence; all where outputs do not go out as pairs.
template <int S>
__device__ __forceinline__ uint32_t odd_tokens(const Span& v, int pairs) {
  constexpr uint32_t all = (1u << S) - 1u;
  const uint32_t odd = __reduce_or_sync(0xffffffffu, (~v.on & all) | v.first | v.last);
  return pairs ? odd : all;
}

// cu == null: sequence b holds [0, T).  cu: sequence n holds [cu[n], cu[n+1]); malformed bounds
// give wrong spans, but never a token outside [0, T) or a sequence outside [0, N).
template <int S>
__device__ __forceinline__ Span span_of(const int* cu, int N, int T, int b, int lo) {
  Span r = {0u, 0u, 0u, b};
  const int hi = min(T, lo + S);
  if (lo >= hi) return r;
  if (!cu) {
    r.on = (1u << (hi - lo)) - 1u;
    if (lo == 0) r.first = 1u;
    if (hi == T) r.last = 1u << (T - 1 - lo);
    return r;
  }
  int l = 0, h = N;  // the first n with cu[n+1] > lo
  while (l < h) {
    const int m = (l + h) >> 1;
    if (cu[m + 1] > lo) h = m;
    else l = m + 1;
  }
  r.n0 = min(l, N - 1);
  for (int n = l; n < N; ++n) {
    const int s = cu[n], e = cu[n + 1];
    if (s >= hi) break;
    if (e <= s) continue;
    if (s >= lo) r.first |= 1u << (s - lo);
    if (e <= hi && e > lo) r.last |= 1u << (e - 1 - lo);
    const int f = max(s, lo) - lo, g = min(e, hi) - lo;
    if (g > f) r.on |= ((1u << (g - f)) - 1u) << f;
  }
  return r;
}

// The sequence after (before) n that is not empty; callers stop at the last (first) themselves.
__device__ __forceinline__ int next_sequence(const int* cu, int N, int n) {
  if (!cu) return n;
  do ++n;
  while (n < N - 1 && cu[n + 1] <= cu[n]);
  return min(n, N - 1);
}
__device__ __forceinline__ int previous_sequence(const int* cu, int n) {
  if (!cu) return n;
  do --n;
  while (n > 0 && cu[n + 1] <= cu[n]);
  return max(n, 0);
}

// ---------------------------------------------------------------- the cluster's scan

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Writes v to p in the shared memory of CTA `rank` of the cluster and counts its 8 bytes on that
// CTA's bar.
__device__ __forceinline__ void send(float2* p, uint64_t* bar, uint32_t rank, float2 v) {
  uint32_t at, b;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(p)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(tc::smem_u32(bar)), "r"(rank));
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at),
      "f"(v.x), "f"(v.y), "r"(b)
      : "memory");
}

struct LinkSmem {
  // the segments' maps; then entry g: that of segments 0 .. g, and the last: the carry into the tile
  float2 seg[kSegs][kCh];
  Span span[kSegs];  // the segments' sequences
  uint64_t bar[2];   // the other tiles' maps are there
  const int* cu;     // the sequences' bounds: here they cost no registers between their uses
};
// The other tiles' maps, of even and odd steps, behind the stages: one per other CTA.
typedef float2 TileMaps[2][kCh];
constexpr size_t maps_bytes(int Z) { return (Z - 1) * sizeof(TileMaps); }
// Bounds of fewer than kManyBounds sequences are read from shared memory, behind the maps: room for
// kManyBounds, or for kFewBounds where these do (1 KB less can be a CTA more per SM: 2500 tokens of
// 514 channels, fp32, backward 22.4 -> 21.4 us).
constexpr int kFewBounds = 16, kManyBounds = 256;
__host__ __device__ __forceinline__ int bounds_room(const GlrArgs& p) {
  return !p.cu || p.N >= kManyBounds ? 0 : p.N < kFewBounds ? kFewBounds : kManyBounds;
}

// Sets sm.cu to the sequences' bounds: a copy at `to`, or where they are.  To be used behind a
// block barrier.
__device__ __forceinline__ void place_bounds(LinkSmem& sm, const GlrArgs& p, void* to) {
  const bool copy = bounds_room(p) != 0;
  if (threadIdx.x == 0) sm.cu = copy ? static_cast<int*>(to) : p.cu;
  if (!copy) return;
  for (int n = threadIdx.x; n <= p.N; n += kThreads) static_cast<int*>(to)[n] = __ldg(p.cu + n);
}

// Before the first step; a barrier over the cluster.
__device__ __forceinline__ void link_init(LinkSmem& sm, int Z) {
  if (Z > 1 && threadIdx.x == 0) {
    tc::mbar_init(&sm.bar[0], 1);
    tc::mbar_init(&sm.bar[1], 1);
    tc::fence_mbar_init();
  }
  __syncthreads();
  if (Z > 1) cluster_sync();
}

// After the segments' maps of step k are in sm.seg: folds them, and moves `c` (warp 0, a channel
// per lane: the carry into the step) on to the next step.  Meanwhile warp 1 looks up the sequences
// of the next step's segments, spans(g): dependent loads of up to 2 us for packed sequences.
// Starts and ends with a block barrier.
//
// A CTA sends its map of step k + 1 after it has read the maps of step k, and has those of step
// k + 1 before it sends that of step k + 2: two buffers are enough.  It leaves the last step
// only with every map that is sent to it in place.
template <typename F>
__device__ __forceinline__ void link_step(LinkSmem& sm, TileMaps* maps, int k, int Z, int rank,
                                          float& c, F spans) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid >= 32 && tid < 32 + kSegs) sm.span[tid - 32] = spans(tid - 32);
  if (tid < kCh) {
    if (Z > 1 && tid == 0)
      tc::mbar_arrive_expect_tx(&sm.bar[k & 1], (Z - 1) * kCh * sizeof(float2));
    float2 m = sm.seg[0][tid];
#pragma unroll
    for (int g = 1; g < kSegs; ++g) {
      then(m, sm.seg[g][tid]);
      if (g < kSegs - 1) sm.seg[g][tid] = m;
    }
    if (Z == 1) {
      sm.seg[kSegs - 1][tid].x = c;
      c = apply(m.x, m.y, c);
    } else {
      for (int z = 0; z < Z; ++z)
        if (z != rank) send(&maps[rank - (rank > z)][k & 1][tid], &sm.bar[k & 1], z, m);
      if (!tc::mbar_wait_short(&sm.bar[k & 1], (k >> 1) & 1)) atomicOr(&g_glr_error, 2u);
      for (int z = 0; z < Z; ++z) {
        if (z == rank) sm.seg[kSegs - 1][tid].x = c;
        const float2 n = z == rank ? m : maps[z - (z > rank)][k & 1][tid];
        c = apply(n.x, n.y, c);
      }
    }
  }
  __syncthreads();
}

// After the last step.  Where a wait ran out of time (only then are maps to this CTA still on their
// way), the CTA stays until all of the cluster have sent theirs and, with a limit again, until they
// are here.  (relaxed: the outputs need no order here, and a release would wait for them)
__device__ __forceinline__ void link_done(LinkSmem& sm, int steps, int Z) {
  if (Z == 1) return;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (int k = max(steps - 2, 0); k < steps && threadIdx.x == 0; ++k)
    tc::mbar_wait_short(&sm.bar[k & 1], (k >> 1) & 1);
}

// The carry into a segment, from the tile's and the segments before it.
__device__ __forceinline__ f32x2 segment_carry(const LinkSmem& sm, int g, int cl) {
  const float4 c = *reinterpret_cast<const float4*>(&sm.seg[kSegs - 1][cl]);
  if (g == 0) return pack(c.x, c.z);
  const float4 m = *reinterpret_cast<const float4*>(&sm.seg[g - 1][cl]);
  return pack(apply(m.x, m.y, c.x), apply(m.z, m.w, c.z));
}

struct Geometry {
  int Z;          // CTAs of a cluster
  int blocks;     // channel blocks
  int pairs;      // the outputs and states can be written two channels at a time
  int x, la, h, dout;  // bytes of a copy (fill)
};

// Sequences without tokens: their state is the one they came with (dst = src, or zero).
__device__ __forceinline__ void empty_sequences(const int* cu, int N, int T, int b, int D, int ch,
                                                int how, const float* src, float* dst) {
  if (!dst) return;
  const int g = threadIdx.x / (kCh / 2);
  const int n0 = cu ? g : (g == 0 && T == 0 ? b : N), step = cu ? kSegs : N;
  for (int n = n0; n < N; n += step) {
    if (cu && cu[n + 1] > cu[n]) continue;
    const int64_t at = (int64_t)n * D + ch;
    store_pair(dst + at, src ? load_state(src + at, how) : make_float2(0.f, 0.f), how);
  }
}

// ---------------------------------------------------------------- forward

template <typename InT, typename GateT, int S>
struct FwdStage {
  Tile<GateT, S> la;
  Tile<InT, S> x;
};

constexpr int kFwdStages = 2;

template <typename InT, typename GateT, typename OutT, int S, int kScale>
__global__ void __launch_bounds__(kThreads, kPerSm) glr_fwd_kernel(GlrArgs p, Geometry geo) {
  constexpr int kRows = kSegs * S;
  using Stage = FwdStage<InT, GateT, S>;
  extern __shared__ __align__(16) uint8_t dyn[];
  Stage* stages = reinterpret_cast<Stage*>(dyn);
  TileMaps* maps = reinterpret_cast<TileMaps*>(stages + kFwdStages);
  __shared__ __align__(16) LinkSmem sm;
  place_bounds(sm, p, maps + geo.Z - 1);
  const int Z = geo.Z, rank = Z > 1 ? (int)cluster_rank() : 0;
  const int item = blockIdx.x / Z, b = item / geo.blocks, blk = item - b * geo.blocks;
  const int seg = threadIdx.x / (kCh / 2);
  const int cl = 2 * (threadIdx.x % (kCh / 2)), ch = blk * kCh + cl;
  const bool live = ch < p.D;
  const int how = ch + 1 >= p.D ? kFirst : geo.pairs ? kPairs : kSingles;
  const int cols = min(kCh, p.D - blk * kCh);
  const InT* x = static_cast<const InT*>(p.x) + b * p.sx[0] + blk * kCh;
  const GateT* la = static_cast<const GateT*>(p.log_a) + b * p.sl[0] + blk * kCh;
  OutT* out = static_cast<OutT*>(p.out) + (int64_t)b * p.T * p.D + ch;
  const int steps = (p.T + Z * kRows - 1) / (Z * kRows);
  auto issue = [&](int k) {
    if (k < steps) {
      Stage& st = stages[k % kFwdStages];
      const int t0 = (k * Z + rank) * kRows, rows = min(kRows, p.T - t0);
      fill(st.la, la + (int64_t)t0 * p.sl[1], p.sl[1], 0, rows, cols, geo.la);
      fill(st.x, x + (int64_t)t0 * p.sx[1], p.sx[1], 0, rows, cols, geo.x);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kFwdStages - 1; ++k) issue(k);
  link_init(sm, Z);
  if (rank == 0 && live) empty_sequences(sm.cu, p.N, p.T, b, p.D, ch, how, p.h0, p.state);
  auto spans = [&](int k, int g) { return span_of<S>(sm.cu, p.N, p.T, b, (k * Z + rank) * kRows + g * S); };
  if (threadIdx.x < kSegs) sm.span[threadIdx.x] = spans(0, threadIdx.x);
  float c = 0.f;
  for (int k = 0; k < steps; ++k) {
    cp_async_wait<kFwdStages - 2>();
    __syncthreads();
    issue(k + kFwdStages - 1);
    const Stage& st = stages[k % kFwdStages];
    const int lo = (k * Z + rank) * kRows + seg * S;
    const Span span = sm.span[seg];
    f32x2 a[S], u[S], A = both(1.f), H = both(0.f);
    const uint32_t odd = odd_tokens<S>(span, geo.pairs);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      f32x2 m;
      gate_of(st.la.pair(seg, s, cl), &a[s], &m);
      u[s] = mul2(scale_of<kScale>(m), to_pair(st.x.pair(seg, s, cl)));
    }
    if (!odd) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        H = fma2(a[s], H, u[s]);
        A = mul2(A, a[s]);
      }
    } else {
      int n = span.n0;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (!(odd >> s & 1)) {
          H = fma2(a[s], H, u[s]);
          A = mul2(A, a[s]);
          continue;
        }
        const bool on = span.on >> s & 1, first = span.first >> s & 1;
        u[s] = on ? u[s] : both(0.f);
        a[s] = on ? a[s] : both(1.f);
        if (p.h0) {
          if (first && live) u[s] = fma2(a[s], to_pair(load_state(p.h0 + (int64_t)n * p.D + ch, how)), u[s]);
          if (span.last >> s & 1) n = next_sequence(sm.cu, p.N, n);
        }
        a[s] = first ? both(-0.f) : a[s];
        A = first ? both(-0.f) : mul2(A, a[s]);
        H = fma2(a[s], first ? both(0.f) : H, u[s]);
      }
    }
    const float2 A1 = unpack(A), H1 = unpack(H);
    *reinterpret_cast<float4*>(&sm.seg[seg][cl]) = make_float4(A1.x, H1.x, A1.y, H1.y);
    keep_products<S>(&sm.seg[seg][cl], A, a);
    link_step(sm, maps, k, Z, rank, c, [&](int g) { return spans(k + 1, g); });
    f32x2 h = segment_carry(sm, seg, cl);
    OutT* o = out + (int64_t)lo * p.D;
    if (!odd) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        h = fma2(a[s], h, u[s]);
        if (live) put_pair(o, unpack(h));
        o += p.D;
      }
    } else {
      int n = span.n0;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (!(odd >> s & 1)) {
          h = fma2(a[s], h, u[s]);
          if (live) put_pair(o, unpack(h));
          o += p.D;
          continue;
        }
        h = fma2(a[s], span.first >> s & 1 ? both(0.f) : h, u[s]);  // (a is -0 there: h = u)
        if (live && (span.on >> s & 1)) store_pair(o, unpack(h), how);
        o += p.D;
        if (p.state && (span.last >> s & 1)) {
          if (live) store_pair(p.state + (int64_t)n * p.D + ch, unpack(h), how);
          n = next_sequence(sm.cu, p.N, n);
        }
      }
    }
    __syncwarp();
  }
  link_done(sm, steps, Z);
}

// ---------------------------------------------------------------- backward
//
// With g_t the gradient of h_t: g_t = dout_t + a_{t+1} g_{t+1} (plus the final state's gradient
// at the end of a sequence), dx_t = b_t g_t, dlog_a_t = a_t h_{t-1} g_t + b'(log a_t) x_t g_t and
// the first state's gradient is a_t g_t at the sequence's first token.  The carry from t to t-1
// is c_t = a_t g_t = a_t c_{t+1} + a_t dout_t, scanned from the end: rank 0's segment 0 holds
// the last S tokens of a step.

template <typename InT, typename GateT, typename GradT, int S, bool kX>
struct BwdStage {
  Tile<GateT, S> la;
  Tile<GradT, S> dout;
  Tile<GradT, S> h;  // of the token before
  Tile<InT, S> x;
};
template <typename InT, typename GateT, typename GradT, int S>
struct BwdStage<InT, GateT, GradT, S, false> {
  Tile<GateT, S> la;
  Tile<GradT, S> dout;
  Tile<GradT, S> h;
};

constexpr int kBwdStages = 2;

template <typename InT, typename GateT, typename GradT, int S, int kScale>
__global__ void __launch_bounds__(kThreads, kPerSm) glr_bwd_kernel(GlrArgs p, Geometry geo) {
  constexpr int kRows = kSegs * S;
  constexpr bool kX = kScale != LL_GLR_NONE;
  using Stage = BwdStage<InT, GateT, GradT, S, kX>;
  extern __shared__ __align__(16) uint8_t dyn[];
  Stage* stages = reinterpret_cast<Stage*>(dyn);
  TileMaps* maps = reinterpret_cast<TileMaps*>(stages + kBwdStages);
  __shared__ __align__(16) LinkSmem sm;
  place_bounds(sm, p, maps + geo.Z - 1);
  const int Z = geo.Z, rank = Z > 1 ? (int)cluster_rank() : 0;
  const int item = blockIdx.x / Z, b = item / geo.blocks, blk = item - b * geo.blocks;
  const int seg = threadIdx.x / (kCh / 2);
  const int cl = 2 * (threadIdx.x % (kCh / 2)), ch = blk * kCh + cl;
  const bool live = ch < p.D;
  const int how = ch + 1 >= p.D ? kFirst : geo.pairs ? kPairs : kSingles;
  const int cols = min(kCh, p.D - blk * kCh);
  const InT* x = static_cast<const InT*>(p.x) + b * p.sx[0] + blk * kCh;
  const GateT* la = static_cast<const GateT*>(p.log_a) + b * p.sl[0] + blk * kCh;
  const int64_t base = (int64_t)b * p.T * p.D + blk * kCh;
  const GradT* dout = static_cast<const GradT*>(p.dout) + base;
  const GradT* hs = static_cast<const GradT*>(p.h) + base;
  GradT* dx = static_cast<GradT*>(p.dx) + base + cl;
  GateT* dla = static_cast<GateT*>(p.dlog_a) + base + cl;
  const int steps = (p.T + Z * kRows - 1) / (Z * kRows);
  // the tile of step k: steps, then ranks, count from the end of the tiles that cover [0, T)
  auto tile_start = [&](int k) { return ((steps - 1 - k) * Z + (Z - 1 - rank)) * kRows; };
  auto issue = [&](int k) {
    if (k < steps) {
      Stage& st = stages[k % kBwdStages];
      const int t0 = tile_start(k), rows = min(kRows, p.T - t0);
      const int64_t at = (int64_t)t0 * p.D;
      fill(st.la, la + (int64_t)t0 * p.sl[1], p.sl[1], 0, rows, cols, geo.la);
      fill(st.dout, dout + at, p.D, 0, rows, cols, geo.dout);
      fill(st.h, hs + at - p.D, p.D, t0 == 0, rows, cols, geo.h);
      if constexpr (kX) fill(st.x, x + (int64_t)t0 * p.sx[1], p.sx[1], 0, rows, cols, geo.x);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kBwdStages - 1; ++k) issue(k);
  link_init(sm, Z);
  if (rank == 0 && live) empty_sequences(sm.cu, p.N, p.T, b, p.D, ch, how, p.dstate, p.dh0);
  auto spans = [&](int k, int g) {
    return span_of<S>(sm.cu, p.N, p.T, b, k < steps ? tile_start(k) + (kSegs - 1 - g) * S : p.T);
  };
  if (threadIdx.x < kSegs) sm.span[threadIdx.x] = spans(0, threadIdx.x);
  float carry = 0.f;
  for (int k = 0; k < steps; ++k) {
    cp_async_wait<kBwdStages - 2>();
    __syncthreads();
    issue(k + kBwdStages - 1);
    const Stage& st = stages[k % kBwdStages];
    const int back = kSegs - 1 - seg, lo = tile_start(k) + back * S;
    const Span span = sm.span[seg];
    int n_last = span.n0;  // the sequence of the last token that is on
    if (p.cu && (p.dstate || p.h0 || p.dh0)) {
#pragma unroll
      for (int s = 0; s < S; ++s)
        if ((span.last >> s & 1) && (span.on >> s) > 1u) n_last = next_sequence(sm.cu, p.N, n_last);
    }
    f32x2 a[S], bs[S], d[S], A = both(1.f), E = both(0.f);
    const uint32_t odd = odd_tokens<S>(span, geo.pairs);
#pragma unroll
    for (int s = S - 1; s >= 0; --s) {
      f32x2 m;
      gate_of(st.la.pair(back, s, cl), &a[s], &m);
      bs[s] = scale_of<kScale>(m);
      d[s] = to_pair(st.dout.pair(back, s, cl));
    }
    if (!odd) {
#pragma unroll
      for (int s = S - 1; s >= 0; --s) {
        A = mul2(A, a[s]);
        E = mul2(a[s], add2(d[s], E));
      }
    } else {
      int n = n_last;
#pragma unroll
      for (int s = S - 1; s >= 0; --s) {
        const bool on = span.on >> s & 1, last = span.last >> s & 1;
        a[s] = on ? a[s] : both(1.f);
        d[s] = on ? d[s] : both(0.f);
        if (p.dstate) {
          if (last && live) d[s] = add2(d[s], to_pair(load_state(p.dstate + (int64_t)n * p.D + ch, how)));
          if (span.first >> s & 1) n = previous_sequence(sm.cu, n);
        }
        A = last ? both(-0.f) : mul2(A, a[s]);  // nothing comes from the sequence behind
        E = mul2(a[s], last ? d[s] : add2(d[s], E));
      }
    }
    const float2 A1 = unpack(A), E1 = unpack(E);
    *reinterpret_cast<float4*>(&sm.seg[seg][cl]) = make_float4(A1.x, E1.x, A1.y, E1.y);
    keep_products<S>(&sm.seg[seg][cl], A, a);
    link_step(sm, maps, k, Z, rank, carry, [&](int g) { return spans(k + 1, g); });
    f32x2 c = segment_carry(sm, seg, cl);
    GradT* ox = dx + (int64_t)(lo + S - 1) * p.D;
    GateT* ol = dla + (int64_t)(lo + S - 1) * p.D;
    if (!odd) {
#pragma unroll
      for (int s = S - 1; s >= 0; --s) {
        const f32x2 g = add2(d[s], c);
        c = mul2(a[s], g);
        f32x2 l = mul2(c, to_pair(st.h.pair(back, s, cl)));
        if constexpr (kX)
          l = fma2(mul2(scale_grad<kScale>(a[s], bs[s]), to_pair(st.x.pair(back, s, cl))), g, l);
        if (live) {
          put_pair(ox, unpack(mul2(bs[s], g)));
          put_pair(ol, unpack(l));
        }
        ox -= p.D;
        ol -= p.D;
      }
    } else {
      int n = n_last;
#pragma unroll
      for (int s = S - 1; s >= 0; --s, ox -= p.D, ol -= p.D) {
        const bool on = span.on >> s & 1, first = span.first >> s & 1;
        const f32x2 g = span.last >> s & 1 ? d[s] : add2(d[s], c);
        f32x2 before = first || lo + s == 0 ? both(0.f) : to_pair(st.h.pair(back, s, cl));
        if (p.h0 && first && live) before = to_pair(load_state(p.h0 + (int64_t)n * p.D + ch, how));
        c = on ? mul2(a[s], g) : c;
        f32x2 l = mul2(c, before);
        if constexpr (kX)
          l = fma2(mul2(scale_grad<kScale>(a[s], bs[s]), to_pair(st.x.pair(back, s, cl))), g, l);
        if (live && on) {
          store_pair(ox, unpack(mul2(bs[s], g)), how);
          store_pair(ol, unpack(l), how);
        }
        if (first && (p.h0 || p.dh0)) {
          if (live && p.dh0) store_pair(p.dh0 + (int64_t)n * p.D + ch, unpack(c), how);
          n = previous_sequence(sm.cu, n);
        }
      }
    }
    __syncwarp();
  }
  link_done(sm, steps, Z);
}

// ---------------------------------------------------------------- step

// One token per row: state[slot] <- a state[slot] + b x, out = the new state.  A slot given
// twice belongs to its first row; the rows after it, and rows whose slot is out of range, are
// left out and raise the error word.  2.1 us for 128 rows of 2048 channels in a graph, the launch
// itself; 12 for 1024 rows of 4096 (67 MB, 5.7 TB/s).
constexpr int kStepThreads = 256;

template <typename InT, typename GateT, typename OutT, int kScale>
__global__ void __launch_bounds__(kStepThreads) glr_step_kernel(
    float* __restrict__ state, const int* __restrict__ slots, int S, const InT* __restrict__ x,
    const GateT* __restrict__ la, OutT* __restrict__ out, int D, int pairs) {
  const int row = blockIdx.y;
  const int ch = (blockIdx.x * kStepThreads + threadIdx.x) * 2;
  const bool on = ch < D;
  const int how = ch + 1 >= D ? kFirst : pairs ? kPairs : kSingles;
  int64_t slot = row;
  float2 xv = make_float2(0.f, 0.f), l = xv;
  const int64_t at = (int64_t)row * D + ch;
  if (on) {
    if (how == kPairs) {
      xv = pair_of(x + at);
      l = pair_of(la + at);
    } else {
      xv.x = to_f32(x[at]);
      l.x = to_f32(la[at]);
      if (how == kSingles) {
        xv.y = to_f32(x[at + 1]);
        l.y = to_f32(la[at + 1]);
      }
    }
  }
  if (slots) {
    const int sl = slots[row];
    bool twice = false;
    for (int r = threadIdx.x; r < row; r += kStepThreads) twice |= slots[r] == sl;
    twice = __syncthreads_or(twice);
    if (sl == -1) return;
    if (sl < 0 || sl >= S || twice) {
      if (threadIdx.x == 0) atomicOr(&g_glr_error, 1u);
      return;
    }
    slot = sl;
  }
  if (!on) return;
  float* st = state + slot * D + ch;
  f32x2 a, m;
  gate_of(l, &a, &m);
  const float2 h = unpack(fma2(a, to_pair(load_state(st, how)), mul2(scale_of<kScale>(m), to_pair(xv))));
  store_pair(st, h, how);
  store_pair(out + at, h, how);
}

// ---------------------------------------------------------------- launch

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Bytes of a copy that pointer, batch stride, row stride and width allow.
int copy_bytes(const void* p, int64_t sb, int64_t st, int64_t D, int size) {
  for (int bytes = 16; bytes >= 4; bytes /= 4) {
    const int per = bytes / size;
    if (per >= 1 && aligned(p, bytes) && sb % per == 0 && st % per == 0 && D % per == 0)
      return bytes;
  }
  return size;
}

struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  Launch(int64_t items, int Z, size_t stages, int bounds, cudaStream_t s) {
    cfg.gridDim = dim3((unsigned)(items * Z));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = stages + maps_bytes(Z) + bounds * sizeof(int);
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = Z;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = Z > 1 ? 1 : 0;
  }
};

// How many clusters of Z CTAs a device holds at once; asked for once per kernel, Z, bounds and
// device (of the first kDevices: the answer takes the runtime longer than the launch).
constexpr int kDevices = 16;
template <auto kKernel>
cudaError_t clusters_held(int dev, int Z, size_t stages, int bounds, int* n) {
  static std::atomic<int> table[kDevices + 1][kMaxCluster + 1][3];
  std::atomic<int>& known = table[std::min(dev, kDevices)][Z][(bounds > 0) + (bounds > kFewBounds)];
  if (dev < kDevices && (*n = known.load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  const Launch l(1, Z, stages, bounds, nullptr);
  const cudaError_t e = cudaOccupancyMaxActiveClusters(n, kKernel, &l.cfg);
  if (e == cudaSuccess) known.store(*n, std::memory_order_relaxed);
  return e;
}

// Z, the CTAs that share a channel block: as many as leave all clusters running at once (at most
// kMaxCluster), then as few as take no more steps.  Forward and backward: 65536 tokens of 512
// channels, bf16, 124 and 230 us with Z = 16, 167 and 316 with 8; 9001 of 1000, fp32, 30 and 45
// with 12, 31 and 49 with 8.  Where a cluster waits for the others: 2500 of 514, fp32, forward 21 us
// with 16 (17 clusters, of which 14 run), 11 with 10 and 15 with 8.
template <auto kKernel>
cudaError_t launch_cluster(const GlrArgs& p, Geometry& g, int rows, size_t stages,
                           cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(stages + maps_bytes(kMaxCluster) + kManyBounds * sizeof(int)));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  const int64_t items = (int64_t)p.B * g.blocks;
  const int tiles = (int)(((int64_t)p.T + rows - 1) / rows);
  g.Z = tiles < 1 ? 1 : tiles < kMaxCluster ? tiles : kMaxCluster;
  const int bounds = bounds_room(p);
  int dev = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  for (; e == cudaSuccess && g.Z > 1; --g.Z) {
    int held = 0;
    e = clusters_held<kKernel>(dev, g.Z, stages, bounds, &held);
    if (items <= held) break;
  }
  if (e != cudaSuccess) return e;
  const int steps = (tiles + g.Z - 1) / g.Z;
  if (steps > 0) g.Z = (tiles + steps - 1) / steps;
  const Launch l(items, g.Z, stages, bounds, s);
  return cudaLaunchKernelEx(&l.cfg, kKernel, p, (const Geometry&)g);
}

template <typename InT, typename GateT, typename OutT, int kScale>
cudaError_t launch(const GlrArgs& p, bool backward, cudaStream_t s) {
  Geometry g;
  g.blocks = (p.D + kCh - 1) / kCh;
  const int64_t dense = (int64_t)p.T * p.D;
  const size_t o = 2 * sizeof(OutT);
  g.pairs = p.D % 2 == 0 && aligned(p.out, o) && aligned(p.state, 8) && aligned(p.dx, o) &&
            aligned(p.dlog_a, 2 * sizeof(GateT)) && aligned(p.dh0, 8);
  g.x = copy_bytes(p.x, p.sx[0], p.sx[1], p.D, sizeof(InT));
  g.la = copy_bytes(p.log_a, p.sl[0], p.sl[1], p.D, sizeof(GateT));
  g.h = copy_bytes(p.h, dense, p.D, p.D, sizeof(OutT));
  g.dout = copy_bytes(p.dout, dense, p.D, p.D, sizeof(OutT));
  if (backward) {
    constexpr int S = 4;  // the backward keeps three values per token in registers
    constexpr size_t stages = kBwdStages * sizeof(BwdStage<InT, GateT, OutT, S, kScale != LL_GLR_NONE>);
    return launch_cluster<glr_bwd_kernel<InT, GateT, OutT, S, kScale>>(p, g, kSegs * S, stages, s);
  }
  constexpr int S = 8;
  constexpr size_t stages = kFwdStages * sizeof(FwdStage<InT, GateT, S>);
  return launch_cluster<glr_fwd_kernel<InT, GateT, OutT, S, kScale>>(p, g, kSegs * S, stages, s);
}

template <typename InT, typename GateT, typename OutT>
cudaError_t launch_scale(const GlrArgs& p, int scale, bool backward, cudaStream_t s) {
  if (scale == LL_GLR_NONE) return launch<InT, GateT, OutT, LL_GLR_NONE>(p, backward, s);
  if (scale == LL_GLR_ONE_MINUS) return launch<InT, GateT, OutT, LL_GLR_ONE_MINUS>(p, backward, s);
  return launch<InT, GateT, OutT, LL_GLR_SQRT>(p, backward, s);
}

template <typename InT, typename GateT, typename OutT, int kScale>
cudaError_t launch_step(float* state, const int* slots, int S, const void* x, const void* la,
                        void* out, int B, int D, cudaStream_t s) {
  const int pairs = D % 2 == 0 && aligned(state, 8) && aligned(x, 2 * sizeof(InT)) &&
                    aligned(la, 2 * sizeof(GateT)) && aligned(out, 2 * sizeof(OutT));
  const dim3 grid((D + 2 * kStepThreads - 1) / (2 * kStepThreads), B);
  glr_step_kernel<InT, GateT, OutT, kScale><<<grid, kStepThreads, 0, s>>>(
      state, slots, S, static_cast<const InT*>(x), static_cast<const GateT*>(la),
      static_cast<OutT*>(out), D, pairs);
  return cudaGetLastError();
}

template <typename InT, typename GateT, typename OutT>
cudaError_t step_scale(float* state, const int* slots, int S, const void* x, const void* la,
                       void* out, int B, int D, int scale, cudaStream_t s) {
  if (scale == LL_GLR_NONE)
    return launch_step<InT, GateT, OutT, LL_GLR_NONE>(state, slots, S, x, la, out, B, D, s);
  if (scale == LL_GLR_ONE_MINUS)
    return launch_step<InT, GateT, OutT, LL_GLR_ONE_MINUS>(state, slots, S, x, la, out, B, D, s);
  return launch_step<InT, GateT, OutT, LL_GLR_SQRT>(state, slots, S, x, la, out, B, D, s);
}

}  // namespace

cudaError_t launch_glr(const GlrArgs& p, int in_dtype, int gate_dtype, int out_dtype, int scale,
                       bool backward, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  const bool o32 = out_dtype == LL_F32;
  if (in_dtype == LL_F32)
    return o32 ? launch_scale<float, float, float>(p, scale, backward, s)
               : launch_scale<float, float, bf16>(p, scale, backward, s);
  if (gate_dtype == LL_F32)
    return o32 ? launch_scale<bf16, float, float>(p, scale, backward, s)
               : launch_scale<bf16, float, bf16>(p, scale, backward, s);
  return o32 ? launch_scale<bf16, bf16, float>(p, scale, backward, s)
             : launch_scale<bf16, bf16, bf16>(p, scale, backward, s);
}

cudaError_t launch_glr_step(float* state, const int* slots, int S, const void* x, const void* la,
                            void* out, int B, int D, int in_dtype, int gate_dtype, int out_dtype,
                            int scale, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  const bool o32 = out_dtype == LL_F32;
  if (in_dtype == LL_F32)
    return o32 ? step_scale<float, float, float>(state, slots, S, x, la, out, B, D, scale, s)
               : step_scale<float, float, bf16>(state, slots, S, x, la, out, B, D, scale, s);
  if (gate_dtype == LL_F32)
    return o32 ? step_scale<bf16, float, float>(state, slots, S, x, la, out, B, D, scale, s)
               : step_scale<bf16, float, bf16>(state, slots, S, x, la, out, B, D, scale, s);
  return o32 ? step_scale<bf16, bf16, float>(state, slots, S, x, la, out, B, D, scale, s)
             : step_scale<bf16, bf16, bf16>(state, slots, S, x, la, out, B, D, scale, s);
}

cudaError_t glr_take_error(cudaStream_t s, unsigned* flags) {
  unsigned v = 0;
  cudaError_t e =
      cudaMemcpyFromSymbolAsync(&v, g_glr_error, sizeof(v), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && v) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbolAsync(g_glr_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  *flags = v;
  return e;
}

}  // namespace ll
