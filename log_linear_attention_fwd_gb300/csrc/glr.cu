// Gated linear recurrence per channel: h_t = a_t h_{t-1} + b_t x_t with a_t = exp(log_a_t) and
// b_t = 1, 1 - a_t or sqrt(1 - a_t^2); its gradients; and its single-token step.
//
// Forward and backward are one scan each.  The maps c -> A c + H of consecutive tokens compose
// to a map of the same form, so a segment of tokens is known by two floats per channel.  A CTA
// takes a tile of 8 * S tokens by 32 * V channels: lane = V adjacent channels, warp = S
// consecutive tokens, whose inputs stay in registers.  Each warp folds its S tokens, the CTA
// folds its 8 warps, publishes the tile's (A, H), folds its predecessors' maps back to the
// first whose carry is final (a decoupled look-back, kLook predecessors at a time), publishes
// its own carry and then runs its tokens once more from the carry, in registers.  Every input
// is read once and every output written once; the published maps add 24 / (8 S) bytes to the
// 8 to 16 bytes an element moves.  The backward is the same scan with time reversed.
//
// Tiles are taken by ticket, oldest time first, so a CTA only ever waits for tiles that are
// already running.  The wait is bounded (kWaitLimitNs): a CTA that gives up raises the device
// error word and publishes zeros, so that the tiles after it do not wait in turn.
//
// A sequence start is a reset: its map ignores the carry.  It is marked by A = -0.0 (a real A
// is never negative), not by A = 0, because 0 * inf would let an overflow of one sequence
// reach the next.
#include <cmath>

#include "ll_internal.cuh"
#include "tc_ptx.cuh"

namespace ll {

// bit 0: a look-back wait ran out of time; bit 1: a step was given a slot that is out of range
// or given twice
__device__ unsigned int g_glr_error = 0;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ---------------------------------------------------------------- element access

// V adjacent elements; V = 2 needs alignment to 2 elements.
template <typename T, int V>
struct Pack;
template <>
struct Pack<float, 1> {
  float r;
  __device__ __forceinline__ void load(const float* p) { r = *p; }
  __device__ __forceinline__ float get(int) const { return r; }
  static __device__ __forceinline__ void store(float* p, const float* v) { *p = v[0]; }
};
template <>
struct Pack<float, 2> {
  float2 r;
  __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ float get(int i) const { return i ? r.y : r.x; }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  }
};
template <>
struct Pack<__nv_bfloat16, 1> {
  __nv_bfloat16 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *p; }
  __device__ __forceinline__ float get(int) const { return __bfloat162float(r); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    *p = __float2bfloat16_rn(v[0]);
  }
};
template <>
struct Pack<__nv_bfloat16, 2> {
  __nv_bfloat162 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = *reinterpret_cast<const __nv_bfloat162*>(p);
  }
  __device__ __forceinline__ float get(int i) const {
    return i ? __high2float(r) : __low2float(r);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v[0], v[1]);
  }
};

// b(log a), and with kGrad its derivative.  The differences from 1 go through expm1: near
// a = 1, where such gates live, 1 - a would lose the digits that a itself still has.
// At a = 1 (log a >= 0) the square root's b is 0 and its infinite derivative is taken as 0.
template <int kScale>
__device__ __forceinline__ float scale_of(float la) {
  if (kScale == LL_GLR_ONE_MINUS) return -expm1f(la);
  if (kScale == LL_GLR_SQRT) return sqrtf(fmaxf(-expm1f(2.f * la), 0.f));
  return 1.f;
}
template <int kScale>
__device__ __forceinline__ float scale_grad(float a, float b) {
  if (kScale == LL_GLR_ONE_MINUS) return -a;
  if (kScale == LL_GLR_SQRT) return b > 0.f ? -a * a / b : 0.f;
  return 0.f;
}

// ---------------------------------------------------------------- maps c -> A c + H

__device__ __forceinline__ float apply(float A, float H, float c) {
  return signbit(A) ? H : fmaf(A, c, H);
}
// (A, H) after (A0, H0), into (A0, H0).
__device__ __forceinline__ void then(float& A0, float& H0, float A, float H) {
  H0 = apply(A, H, H0);
  A0 = signbit(A) || signbit(A0) ? -0.f : A * A0;
}

// ---------------------------------------------------------------- sequences

// The sequences of tokens [lo, lo + S): bit i of first / last: token lo + i begins / ends its
// sequence; of on: it belongs to one.  n0: the sequence that holds the first token that is on.
struct Span {
  uint32_t first, last, on;
  int n0;
};

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
    if (__ldg(cu + m + 1) > lo) h = m;
    else l = m + 1;
  }
  r.n0 = min(l, N - 1);
  for (int n = l; n < N; ++n) {
    const int s = __ldg(cu + n), e = __ldg(cu + n + 1);
    if (s >= hi) break;
    if (e <= s) continue;
    if (s >= lo) r.first |= 1u << (s - lo);
    if (e <= hi && e > lo) r.last |= 1u << (e - 1 - lo);
    for (int t = max(s, lo); t < min(e, hi); ++t) r.on |= 1u << (t - lo);
  }
  return r;
}

// The sequence after n that is not empty (callers stop at the last one themselves).
__device__ __forceinline__ int next_sequence(const int* cu, int N, int n) {
  if (!cu) return n;
  do ++n;
  while (n < N - 1 && __ldg(cu + n + 1) <= __ldg(cu + n));
  return min(n, N - 1);
}
__device__ __forceinline__ int previous_sequence(const int* cu, int n) {
  if (!cu) return n;
  do --n;
  while (n > 0 && __ldg(cu + n + 1) <= __ldg(cu + n));
  return max(n, 0);
}

// ---------------------------------------------------------------- look-back

constexpr int kAgg = 1, kFinal = 2;  // flag values: the tile's map, and also its carry

__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Waits until a tile has published something; 0 if it does not within the limit.
__device__ __forceinline__ uint32_t wait_flag(const uint32_t* p) {
  uint32_t v = load_acquire(p);
  if (v) return v;
  const uint64_t t0 = tc::global_timer_ns();
  while (!(v = load_acquire(p)))
    if (tc::global_timer_ns() - t0 > tc::kWaitLimitNs) return 0;
  return v;
}

struct Link {
  float* A;          // [tiles][CH] the tiles' maps and
  float* H;
  float* C;          // final carries, of this batch entry and channel block
  uint32_t* flags;   // [tiles]
};

template <int CH>
struct LinkSmem {
  float A[kWarps][CH], H[kWarps][CH];  // the warps' maps
  float lA[kThreads / CH][CH], lH[kThreads / CH][CH];
  float carry[CH];
  uint32_t flag[kThreads / CH];
  uint32_t ticket;
};

// The carry into tile i: publishes the tile's map, folds the predecessors' and publishes the
// tile's own carry.  Leaves the carry in sm.carry.  All threads call it, after the warps' maps
// are in sm.A and sm.H (no barrier in between needed).
template <int CH>
__device__ __forceinline__ void link_tile(LinkSmem<CH>& sm, const Link& k, int i, int tiles) {
  constexpr int kLook = kThreads / CH;
  const int tid = threadIdx.x, ch = tid % CH, grp = tid / CH;
  float A = 1.f, H = 0.f;
  __syncthreads();
  if (tid < CH) {
    A = sm.A[0][ch];
    H = sm.H[0][ch];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) then(A, H, sm.A[w][ch], sm.H[w][ch]);
    if (i == 0) sm.carry[ch] = 0.f;
    if (tiles > 1) {
      if (i == 0) {
        __stcg(k.C + ch, apply(A, H, 0.f));
      } else {
        __stcg(k.A + (int64_t)i * CH + ch, A);
        __stcg(k.H + (int64_t)i * CH + ch, H);
      }
    }
  }
  __syncthreads();
  if (tiles == 1) return;
  if (tid == 0) store_release(k.flags + i, i == 0 ? kFinal : kAgg);
  if (i == 0) return;
  // the predecessors i-1, i-2, ... in groups of kLook, nearest first
  float bA = 1.f, bH = 0.f;  // (threads below CH) the map of what has been folded so far
  for (int top = i - 1;; top -= kLook) {
    const int j = top - grp;
    if (ch == 0) {
      uint32_t f = kFinal;
      if (j >= 0 && !(f = wait_flag(k.flags + j))) {
        atomicOr(&g_glr_error, 1u);
        f = 3u;
      }
      sm.flag[grp] = f;
    }
    __syncthreads();
    const uint32_t f = sm.flag[grp];
    float a = -0.f, h = 0.f;
    if (j >= 0 && f != 3u) {
      if (f == kFinal) {
        h = __ldcg(k.C + (int64_t)j * CH + ch);
      } else {
        a = __ldcg(k.A + (int64_t)j * CH + ch);
        h = __ldcg(k.H + (int64_t)j * CH + ch);
      }
    }
    sm.lA[grp][ch] = a;
    sm.lH[grp][ch] = h;
    bool done = false;
#pragma unroll
    for (int g = 0; g < kLook; ++g) done |= sm.flag[g] != kAgg;
    __syncthreads();
    if (tid < CH) {
#pragma unroll
      for (int g = 0; g < kLook; ++g) {  // the map so far comes after the farther one
        float fA = sm.lA[g][ch], fH = sm.lH[g][ch];
        then(fA, fH, bA, bH);
        bA = fA;
        bH = fH;
      }
    }
    if (done) break;
  }
  if (tid < CH) {
    const float c = bH;  // a final carry resets, so nothing before it is left in bA
    sm.carry[ch] = c;
    __stcg(k.C + (int64_t)i * CH + ch, apply(A, H, c));
  }
  __syncthreads();
  if (tid == 0) store_release(k.flags + i, kFinal);
}

// The carry into warp w's tokens, from the tile's and the warps before it.
template <int CH>
__device__ __forceinline__ float warp_carry(const LinkSmem<CH>& sm, int w, int ch) {
  float c = sm.carry[ch];
  for (int u = 0; u < w; ++u) c = apply(sm.A[u][ch], sm.H[u][ch], c);
  return c;
}

struct Geometry {
  int tiles, blocks;  // tiles of time, blocks of channels
  float* agg;         // [3][B][blocks][tiles][CH]
  uint32_t* flags;    // [B][blocks][tiles], then the ticket
};

// This CTA's tile (time, channel block, batch entry), by ticket.
template <int CH>
__device__ __forceinline__ void take_tile(LinkSmem<CH>& sm, const Geometry& g, int B, int* i,
                                          int* blk, int* b) {
  const int per = g.blocks * B;
  uint32_t ticket = blockIdx.x;
  if (g.tiles > 1) {
    if (threadIdx.x == 0) sm.ticket = atomicAdd(g.flags + (int64_t)g.tiles * per, 1u);
    __syncthreads();
    ticket = sm.ticket;
  }
  *i = ticket / per;
  const int rest = ticket - *i * per;
  *b = rest / g.blocks;
  *blk = rest - *b * g.blocks;
}

template <int CH>
__device__ __forceinline__ Link link_of(const Geometry& g, int B, int blk, int b) {
  const int64_t line = (int64_t)b * g.blocks + blk, all = (int64_t)B * g.blocks * g.tiles * CH;
  Link k;
  k.A = g.agg + line * g.tiles * CH;
  k.H = k.A + all;
  k.C = k.H + all;
  k.flags = g.flags + line * g.tiles;
  return k;
}

// Sequences without tokens: their state is the one they came with (dst = src, or zero).
template <int V>
__device__ __forceinline__ void empty_sequences(const int* cu, int N, int T, int b, int D, int ch,
                                                const float* src, float* dst) {
  if (!dst || ch >= D) return;
  const int w = threadIdx.x >> 5;
  const int n0 = cu ? w : (w == 0 && T == 0 ? b : N), step = cu ? kWarps : N;
  for (int n = n0; n < N; n += step) {
    if (cu && __ldg(cu + n + 1) > __ldg(cu + n)) continue;
    for (int v = 0; v < V; ++v)
      dst[(int64_t)n * D + ch + v] = src ? src[(int64_t)n * D + ch + v] : 0.f;
  }
}

// ---------------------------------------------------------------- forward

template <typename InT, typename GateT, typename OutT, int V, int S, int kScale>
__global__ void __launch_bounds__(kThreads, 2) glr_fwd_kernel(GlrArgs p, Geometry geo) {
  constexpr int CH = 32 * V;
  __shared__ LinkSmem<CH> sm;
  int i, blk, b;
  take_tile(sm, geo, p.B, &i, &blk, &b);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int cl = lane * V, ch = blk * CH + cl;
  const int lo = (i * kWarps + w) * S;
  const bool live = ch < p.D;
  const InT* x = static_cast<const InT*>(p.x) + b * p.sx[0] + ch;
  const GateT* la = static_cast<const GateT*>(p.log_a) + b * p.sl[0] + ch;
  Pack<InT, V> xr[S];
  Pack<GateT, V> lr[S];
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (live && lo + s < p.T) {
      lr[s].load(la + (int64_t)(lo + s) * p.sl[1]);
      xr[s].load(x + (int64_t)(lo + s) * p.sx[1]);
    }
  const Span span = span_of<S>(p.cu, p.N, p.T, b, lo);
  if (i == 0) empty_sequences<V>(p.cu, p.N, p.T, b, p.D, ch, p.h0, p.state);
  float a[S][V], u[S][V], A[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.f;
    H[v] = 0.f;
  }
  int n = span.n0;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const bool on = live && (span.on >> s & 1);
    const bool first = span.first >> s & 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float l = on ? lr[s].get(v) : 0.f;
      a[s][v] = expf(l);
      u[s][v] = on ? scale_of<kScale>(l) * xr[s].get(v) : 0.f;
    }
    if (first) {
      if (on && p.h0) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          u[s][v] = fmaf(a[s][v], p.h0[(int64_t)n * p.D + ch + v], u[s][v]);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) a[s][v] = -0.f;
    }
    if (span.last >> s & 1) n = next_sequence(p.cu, p.N, n);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      H[v] = apply(a[s][v], u[s][v], H[v]);
      A[v] *= a[s][v];
      if (first) A[v] = -0.f;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sm.A[w][cl + v] = A[v];
    sm.H[w][cl + v] = H[v];
  }
  link_tile<CH>(sm, link_of<CH>(geo, p.B, blk, b), i, geo.tiles);
  if (!live) return;
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = warp_carry<CH>(sm, w, cl + v);
  OutT* out = static_cast<OutT*>(p.out) + ((int64_t)b * p.T + lo) * p.D + ch;
  n = span.n0;
#pragma unroll
  for (int s = 0; s < S; ++s) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = apply(a[s][v], u[s][v], h[v]);
    if (span.on >> s & 1) Pack<OutT, V>::store(out + (int64_t)s * p.D, h);
    if (span.last >> s & 1) {
      if (p.state) Pack<float, V>::store(p.state + (int64_t)n * p.D + ch, h);
      n = next_sequence(p.cu, p.N, n);
    }
  }
}

// ---------------------------------------------------------------- backward
//
// With g_t the gradient of h_t: g_t = dout_t + a_{t+1} g_{t+1} (plus the final state's gradient
// at the end of a sequence), dx_t = b_t g_t, dlog_a_t = a_t h_{t-1} g_t + b'(log a_t) x_t g_t and
// the first state's gradient is a_t g_t at the sequence's first token.  The carry from t to t-1
// is c_t = a_t g_t = a_t c_{t+1} + a_t dout_t, scanned with tile 0 the last in time.

template <typename InT, typename GateT, typename GradT, int V, int S, int kScale>
__global__ void __launch_bounds__(kThreads, 2) glr_bwd_kernel(GlrArgs p, Geometry geo) {
  constexpr int CH = 32 * V;
  constexpr bool kX = kScale != LL_GLR_NONE;
  __shared__ LinkSmem<CH> sm;
  int i, blk, b;
  take_tile(sm, geo, p.B, &i, &blk, &b);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int cl = lane * V, ch = blk * CH + cl;
  // warp w holds the w-th segment from the tile's end
  const int lo = ((geo.tiles - 1 - i) * kWarps + (kWarps - 1 - w)) * S;
  const bool live = ch < p.D;
  const InT* x = static_cast<const InT*>(p.x) + b * p.sx[0] + ch;
  const GateT* la = static_cast<const GateT*>(p.log_a) + b * p.sl[0] + ch;
  const int64_t at = ((int64_t)b * p.T + lo) * p.D + ch;
  const GradT* dout = static_cast<const GradT*>(p.dout) + at;
  const GradT* hs = static_cast<const GradT*>(p.h) + at;
  Pack<InT, V> xr[S];
  Pack<GateT, V> lr[S];
  Pack<GradT, V> gr[S], hr[S];  // hr[s]: h of the token before lo + s
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (live && lo + s < p.T) {
      lr[s].load(la + (int64_t)(lo + s) * p.sl[1]);
      gr[s].load(dout + (int64_t)s * p.D);
    }
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (live && lo + s < p.T) {
      if (lo + s > 0) hr[s].load(hs + (int64_t)(s - 1) * p.D);
      if (kX) xr[s].load(x + (int64_t)(lo + s) * p.sx[1]);
    }
  const Span span = span_of<S>(p.cu, p.N, p.T, b, lo);
  if (i == 0) empty_sequences<V>(p.cu, p.N, p.T, b, p.D, ch, p.dstate, p.dh0);
  // the sequence of the last token that is on
  int n_last = span.n0;
#pragma unroll
  for (int s = 0; s < S; ++s)
    if ((span.last >> s & 1) && (span.on >> s) > 1u) n_last = next_sequence(p.cu, p.N, n_last);
  float A[V], E[V], a[S][V], d[S][V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.f;
    E[v] = 0.f;
  }
  int n = n_last;
#pragma unroll
  for (int s = S - 1; s >= 0; --s) {
    const bool on = live && (span.on >> s & 1);
    const bool last = span.last >> s & 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      a[s][v] = on ? expf(lr[s].get(v)) : 1.f;
      d[s][v] = on ? gr[s].get(v) : 0.f;
    }
    if (last && on && p.dstate) {
#pragma unroll
      for (int v = 0; v < V; ++v) d[s][v] += p.dstate[(int64_t)n * p.D + ch + v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      E[v] = a[s][v] * (last ? d[s][v] : d[s][v] + E[v]);
      A[v] = last ? -0.f : A[v] * a[s][v];
    }
    if (span.first >> s & 1) n = previous_sequence(p.cu, n);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sm.A[w][cl + v] = A[v];
    sm.H[w][cl + v] = E[v];
  }
  link_tile<CH>(sm, link_of<CH>(geo, p.B, blk, b), i, geo.tiles);
  if (!live) return;
  float c[V];
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = warp_carry<CH>(sm, w, cl + v);
  GradT* dx = static_cast<GradT*>(p.dx) + at;
  GateT* dla = static_cast<GateT*>(p.dlog_a) + at;
  n = n_last;
#pragma unroll
  for (int s = S - 1; s >= 0; --s) {
    if (!(span.on >> s & 1)) continue;
    const bool last = span.last >> s & 1, first = span.first >> s & 1;
    float ox[V], ol[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float g = last ? d[s][v] : d[s][v] + c[v];
      const float before =
          first ? (p.h0 ? p.h0[(int64_t)n * p.D + ch + v] : 0.f) : (lo + s > 0 ? hr[s].get(v) : 0.f);
      const float bs = scale_of<kScale>(lr[s].get(v));
      c[v] = a[s][v] * g;
      ox[v] = bs * g;
      ol[v] = c[v] * before;
      if (kX) ol[v] = fmaf(scale_grad<kScale>(a[s][v], bs) * xr[s].get(v), g, ol[v]);
    }
    Pack<GradT, V>::store(dx + (int64_t)s * p.D, ox);
    Pack<GateT, V>::store(dla + (int64_t)s * p.D, ol);
    if (first) {
      if (p.dh0) Pack<float, V>::store(p.dh0 + (int64_t)n * p.D + ch, c);
      n = previous_sequence(p.cu, n);
    }
  }
}

// ---------------------------------------------------------------- step

// One token per row: state[slot] <- a state[slot] + b x, out = the new state.  A slot given
// twice belongs to its first row; the rows after it, and rows whose slot is out of range, are
// left out and raise the error word.
template <typename InT, typename GateT, typename OutT, int V, int kScale>
__global__ void __launch_bounds__(kThreads) glr_step_kernel(
    float* __restrict__ state, const int* __restrict__ slots, int S, const InT* __restrict__ x,
    const GateT* __restrict__ la, OutT* __restrict__ out, int D) {
  const int row = blockIdx.y;
  const int ch = (blockIdx.x * kThreads + threadIdx.x) * V;
  int64_t slot = row;
  const bool on = ch < D;
  Pack<InT, V> xr;
  Pack<GateT, V> lr;
  const int64_t at = (int64_t)row * D + ch;
  if (on) {
    xr.load(x + at);
    lr.load(la + at);
  }
  if (slots) {
    const int sl = slots[row];
    bool twice = false;
    for (int r = threadIdx.x; r < row; r += kThreads) twice |= slots[r] == sl;
    twice = __syncthreads_or(twice);
    if (sl == -1) return;
    if (sl < 0 || sl >= S || twice) {
      if (threadIdx.x == 0) atomicOr(&g_glr_error, 2u);
      return;
    }
    slot = sl;
  }
  if (!on) return;
  float* st = state + slot * D + ch;
  Pack<float, V> h0;
  h0.load(st);
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float l = lr.get(v);
    h[v] = fmaf(expf(l), h0.get(v), scale_of<kScale>(l) * xr.get(v));
  }
  Pack<float, V>::store(st, h);
  Pack<OutT, V>::store(out + at, h);
}

// ---------------------------------------------------------------- launch

constexpr int kSteps = 8;  // tokens a warp holds

int tiles_of(int64_t T) {
  const int64_t t = (T + kWarps * kSteps - 1) / (kWarps * kSteps);
  return (int)(t < 1 ? 1 : t);
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Channels two at a time wherever pointers and strides allow it.
bool pairs_ok(const GlrArgs& p, int in_size, int gate_size, int out_size) {
  auto ok = [](const void* q, size_t a) { return reinterpret_cast<uintptr_t>(q) % a == 0; };
  return p.D % 2 == 0 && p.sx[0] % 2 == 0 && p.sx[1] % 2 == 0 && p.sl[0] % 2 == 0 &&
         p.sl[1] % 2 == 0 && ok(p.x, 2 * in_size) && ok(p.log_a, 2 * gate_size) &&
         ok(p.dlog_a, 2 * gate_size) && ok(p.out, 2 * out_size) && ok(p.h, 2 * out_size) &&
         ok(p.dout, 2 * out_size) && ok(p.dx, 2 * out_size) && ok(p.h0, 8) && ok(p.state, 8) &&
         ok(p.dstate, 8) && ok(p.dh0, 8);
}

template <typename InT, typename GateT, typename OutT, int V, int kScale>
cudaError_t launch(const GlrArgs& p, bool backward, void* ws, cudaStream_t s) {
  constexpr int CH = 32 * V;
  Geometry g;
  g.tiles = tiles_of(p.T);
  g.blocks = (p.D + CH - 1) / CH;
  const size_t lines = (size_t)p.B * g.blocks * g.tiles;
  g.agg = static_cast<float*>(ws);
  g.flags = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + align256(lines * CH * 12));
  if (g.tiles > 1) {
    const cudaError_t e = cudaMemsetAsync(g.flags, 0, (lines + 1) * sizeof(uint32_t), s);
    if (e != cudaSuccess) return e;
  }
  if (backward)
    glr_bwd_kernel<InT, GateT, OutT, V, kSteps, kScale><<<(unsigned)lines, kThreads, 0, s>>>(p, g);
  else
    glr_fwd_kernel<InT, GateT, OutT, V, kSteps, kScale><<<(unsigned)lines, kThreads, 0, s>>>(p, g);
  return cudaGetLastError();
}

template <typename InT, typename GateT, typename OutT, int kScale>
cudaError_t launch_v(const GlrArgs& p, bool backward, void* ws, cudaStream_t s) {
  return pairs_ok(p, sizeof(InT), sizeof(GateT), sizeof(OutT))
             ? launch<InT, GateT, OutT, 2, kScale>(p, backward, ws, s)
             : launch<InT, GateT, OutT, 1, kScale>(p, backward, ws, s);
}

template <typename InT, typename GateT, typename OutT>
cudaError_t launch_scale(const GlrArgs& p, int scale, bool backward, void* ws, cudaStream_t s) {
  if (scale == LL_GLR_NONE) return launch_v<InT, GateT, OutT, LL_GLR_NONE>(p, backward, ws, s);
  if (scale == LL_GLR_ONE_MINUS)
    return launch_v<InT, GateT, OutT, LL_GLR_ONE_MINUS>(p, backward, ws, s);
  return launch_v<InT, GateT, OutT, LL_GLR_SQRT>(p, backward, ws, s);
}

template <typename InT, typename GateT, typename OutT, int kScale>
cudaError_t launch_step(float* state, const int* slots, int S, const void* x, const void* la,
                        void* out, int B, int D, cudaStream_t s) {
  auto ok = [](const void* q, size_t a) { return reinterpret_cast<uintptr_t>(q) % a == 0; };
  const bool two = D % 2 == 0 && ok(state, 8) && ok(x, 2 * sizeof(InT)) &&
                   ok(la, 2 * sizeof(GateT)) && ok(out, 2 * sizeof(OutT));
  const int per = kThreads * (two ? 2 : 1);
  const dim3 grid((D + per - 1) / per, B);
  const InT* xi = static_cast<const InT*>(x);
  const GateT* lg = static_cast<const GateT*>(la);
  OutT* o = static_cast<OutT*>(out);
  if (two)
    glr_step_kernel<InT, GateT, OutT, 2, kScale>
        <<<grid, kThreads, 0, s>>>(state, slots, S, xi, lg, o, D);
  else
    glr_step_kernel<InT, GateT, OutT, 1, kScale>
        <<<grid, kThreads, 0, s>>>(state, slots, S, xi, lg, o, D);
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

// Sized for the widest form (one channel per lane), whichever the call takes.
int64_t glr_tiles(int64_t B, int64_t T, int64_t D) { return B * ((D + 31) / 32) * tiles_of(T); }

size_t glr_workspace_bytes(int64_t B, int64_t T, int64_t D) {
  if (tiles_of(T) <= 1) return 0;
  const size_t lines = (size_t)glr_tiles(B, T, D);
  return align256(lines * 64 * 12) + align256((lines + 1) * sizeof(uint32_t));
}

cudaError_t launch_glr(const GlrArgs& p, int in_dtype, int gate_dtype, int out_dtype, int scale,
                       bool backward, void* ws, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  const bool o32 = out_dtype == LL_F32;
  if (in_dtype == LL_F32)
    return o32 ? launch_scale<float, float, float>(p, scale, backward, ws, s)
               : launch_scale<float, float, bf16>(p, scale, backward, ws, s);
  if (gate_dtype == LL_F32)
    return o32 ? launch_scale<bf16, float, float>(p, scale, backward, ws, s)
               : launch_scale<bf16, float, bf16>(p, scale, backward, ws, s);
  return o32 ? launch_scale<bf16, bf16, float>(p, scale, backward, ws, s)
             : launch_scale<bf16, bf16, bf16>(p, scale, backward, ws, s);
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
