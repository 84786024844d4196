// Verification of a tree of drafted tokens against the target's probabilities (speculative
// sampling), from given random numbers.
//
// The walk starts at node 0, the pending token, and tries the current node's children in the order of their
// index, against what is left of the target's distribution P there: R_0 = P, Z_0 = 1.  A child with
// token x and random number u is accepted where
//     u Z_k < R_k(x)              (drafts that were given: x is removed from R when it is rejected)
//     u Z_k q(x) < R_k(x)         (drafts drawn from q: then R_{k+1} = max(R_k - Z_k q, 0), Z_{k+1} = sum of it)
// and else the next one is tried; where none is left the next token is drawn from R_k.  So the
// tokens are distributed as the target's own, where its rows sum to 1.  R_k is max(P - S_k q, 0) with S_k = Z_0 + .. + Z_{k-1}, as
// what has once reached 0 stays there: one product per value, whatever was rejected before.
//
// Sums over a vocabulary are 64-bit fixed point with 43 fractional bits: the same in every order, so
// the token drawn depends on no launch shape.  fp32 sums would move the boundaries between 1e5 tokens by
// more than the tokens' own width; fp64 runs at 1/64 of fp32's rate here.
//
// A cluster serves a row, each warp of it a run of the vocabulary.  All CTAs walk alike, from the
// children's values in shared memory; a pass over the vocabulary (one per rejection of a drawn draft, one at the
// end of the walk otherwise) reads the row or two rows once and leaves a sum per warp, and the run that
// holds the drawn token is read again.
//
// Measured (GB300, calls in a row; floor: bytes at the measured copy rate).  One row of 32768 fp32 values: 7.4 us, a
// chain of five latencies (tree, children's values, pass, cluster, run).  61 rows of 131072 with trees of 32: 15 us, 32 MB,
// floor 4.8: the same chain; the pass (4 us) is the only part that moves bytes.  128 chains of 5 drawn drafts: 33 us,
// 134 MB, floor 20: one pass per row (a chain's node has no sibling to try behind a rejection), all rows at once and in step, so
// that nothing moves before the pass and during the search behind it.  32 trees of 23 drawn drafts, 50021 bf16
// values: 30 us, one pass per rejection, each about 2 us of latency and of arithmetic.  Four CTAs of 256
// threads per SM: three left the drawn chains at 54, two of 512 were slower on two of these.
#include <algorithm>

#include "cache_common.cuh"

namespace ll {
namespace {

__device__ unsigned g_verify_error;

constexpr int kNodes = LL_TREE_MAX;
constexpr int kFraction = 43;
constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifySplit = 8;  // CTAs of a cluster
typedef unsigned long long Mass;
constexpr Mass kOne = 1ull << kFraction;
constexpr Mass kMost = (1ull << 62) - 1;  // what S counts as at most, nearly 2^19: its products need 62 bits

// x in [0, 1] (below and NaN: 0, above: 1) as fixed point, to the nearest, plus kBias.  A sum with 8
// has x's first 20 fractional bits as its last ones, and what is left plus 2^-20 the next 23.
constexpr Mass kBias = ((Mass)0x41000000u << 23) + 0x35800000u;
__device__ __forceinline__ Mass biased_mass(float x) {  // x in [0, 1]
  const float hi = __fadd_rz(x, 8.f);
  const float lo = __fadd_rn(__fsub_rn(x, __fsub_rn(hi, 8.f)), 0x1p-20f);
  return (Mass)__float_as_uint(hi) * (1u << 23) + __float_as_uint(lo);
}
__device__ __forceinline__ Mass to_mass(float x) { return biased_mass(__saturatef(x)) - kBias; }
// floor(s x), x as above, for s < 2^62.
__device__ __forceinline__ Mass mass_times(Mass s, float x) {
  const unsigned b = __float_as_uint(__saturatef(x)), m = (b & 0x7fffffu) | 0x800000u;
  const Mass lo = (s & 0xffffffffu) * m, hi = (s >> 32) * m + (lo >> 32);  // s m = hi 2^32 + low word of lo
  const Mass y = hi << 9 | (lo & 0xffffffffu) >> 23;                        // s times the significand
  return y >> min(127u - (b >> 23), 63u);
}
__device__ __forceinline__ Mass less(Mass p, Mass q) { return p > q ? p - q : 0; }

struct VerifyArgs {
  const int* parents;
  const int* tokens;
  const void* probs;
  const void* draft;  // may be null
  const float* u;
  int* path;
  int* count;
  int* token;
  int N, split;
  int64_t V;
};

template <typename T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);
  uint4 w;
  __device__ __forceinline__ float at(int i) const {
    const uint32_t x = (&w.x)[sizeof(T) == 2 ? i >> 1 : i];
    return __uint_as_float(sizeof(T) == 4 ? x : i & 1 ? x & 0xffff0000u : x << 16);
  }
};

// What is drawn from: P alone (kPlain), max(P - Q, 0) (kFirst) or max(P - S Q, 0) (kMore), added to sum.
enum Kind { kPlain, kFirst, kMore };
template <int kKind>
__device__ __forceinline__ void add_rest(Mass& sum, float p, float q, Mass S) {
  if (kKind == kPlain) {
    sum += to_mass(p);
  } else if (kKind == kFirst) {  // (the biases cancel; rounding keeps the order)
    p = __saturatef(p);
    q = __saturatef(q);
    if (p > q) sum += biased_mass(p) - biased_mass(q);
  } else {
    sum += less(to_mass(p), mass_times(S, q));
  }
}
template <int kKind>
__device__ __forceinline__ Mass rest_of(float p, float q, Mass S) {
  Mass sum = 0;
  add_rest<kKind>(sum, p, q, S);
  return sum;
}

// The calling warp's sum over [lo, hi) of a row.  vec: the two rows lie alike to 16 bytes, `off` elements behind one.
template <typename T, int kKind>
__device__ __forceinline__ Mass sum_run(const T* P, const T* Q, int64_t lo, int64_t hi, bool vec, int off, Mass S) {
  constexpr int n = Vec<T>::n, kFlight = kKind == kPlain ? 8 : kKind == kFirst ? 4 : 2;  // loads on their way
  const int lane = threadIdx.x & 31;
  int64_t a = hi, b = hi;  // whole vectors: [a, b)
  if (vec) {
    a = min(hi, ((lo + off + n - 1) & ~(int64_t)(n - 1)) - off);
    b = max(a, ((hi + off) & ~(int64_t)(n - 1)) - off);
  }
  Mass sum = 0;
  auto one = [&](int64_t x) { add_rest<kKind>(sum, to_f32(P[x]), kKind == kPlain ? 0.f : to_f32(Q[x]), S); };
#pragma unroll 1
  for (int64_t x = lo + lane; x < a; x += 32) one(x);
#pragma unroll 1
  for (int64_t x = b + lane; x < hi; x += 32) one(x);
#pragma unroll 1
  for (int64_t x0 = a + lane * n; x0 < b; x0 += 32 * n * kFlight) {
    Vec<T> p[kFlight], q[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int64_t x = x0 + u * 32 * n;
      p[u].w = q[u].w = make_uint4(0u, 0u, 0u, 0u);
      if (x < b) {
        p[u].w = __ldg(reinterpret_cast<const uint4*>(P + x));
        if (kKind != kPlain) q[u].w = __ldg(reinterpret_cast<const uint4*>(Q + x));
      }
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
#pragma unroll
      for (int i = 0; i < n; ++i) add_rest<kKind>(sum, p[u].at(i), kKind == kPlain ? 0.f : q[u].at(i), S);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum;
}

// A function of its own: registers of the loop that has most to do (128 chains of drawn drafts 37 -> 33 us).
template <typename T>
__device__ __noinline__ Mass sum_first(const T* P, const T* Q, int64_t lo, int64_t hi, bool vec, int off) {
  return sum_run<T, kFirst>(P, Q, lo, hi, vec, off, kOne);
}

struct VerifySmem {
  int up[kNodes], tok[kNodes];
  float px[kNodes], qx[kNodes], us[kNodes];
  Mass rest[kNodes];         // drafts that were given: R of a child at its turn
  unsigned first[2], ok[2];  // theirs, a bit per node: no earlier sibling has its token; accepted at its turn
  Mass warp_sum[2][kVerifyWarps], part[kVerifyWarps], scan[kVerifyWarps];  // warp_sum, cta_sum: by turns, as a warp may be
  Mass cta_sum[2][kVerifySplit];                       // at the next pass while another reads the last one's
};

__device__ __forceinline__ void store_remote(Mass* p, uint32_t rank, Mass v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

// As cluster_arrive, but orders no memory.
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

// grid: row, CTA of its cluster (fastest).  kDrawn: with the draft's distributions.
template <typename T, bool kDrawn>
__global__ void __launch_bounds__(kVerifyThreads, 4) tree_verify_kernel(VerifyArgs a) {
  __shared__ VerifySmem sm;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, N = a.N;
  const int C = a.split, rank = blockIdx.x % C;
  const int64_t V = a.V, row = blockIdx.x / C;
  const T* P0 = static_cast<const T*>(a.probs) + row * N * V;
  const T* Q0 = kDrawn ? static_cast<const T*>(a.draft) + row * N * V : nullptr;
  if (C > 1) cluster_arrive_relaxed();  // this CTA is there
  bool bad = false;
  if (tid < kNodes) {
    int up = -2, x = 0;
    if (tid < N) {
      up = a.parents[row * N + tid];
      x = a.tokens[row * N + tid];
      sm.us[tid] = fminf(fmaxf(a.u[row * N + tid], 0.f), 0x1.fffffep-1f);
    }
    const bool child = up >= 0 && up < tid;
    bad = child ? x < 0 || x >= V : up != -1 && up != -2;
    if (bad) up = -2;
    sm.up[tid] = up;
    sm.tok[tid] = x;
    if (up >= 0) {
      sm.px[tid] = to_f32(P0[up * V + x]);
      if (kDrawn) sm.qx[tid] = to_f32(Q0[up * V + x]);
    }
  }
  __syncthreads();
  // drafts that were given: a child's turn comes when all earlier siblings have been rejected, so R and Z there
  // are known from the start: R is 0 where one of those has its token, Z what their R leave
  int up = -2;
  if (tid < kNodes) {
    up = sm.up[tid];
    if (up >= 0) bad |= sm.up[up] == -2;
    if (!kDrawn) {
      const int x = sm.tok[tid];
      bool first = up >= 0;
      for (int i = 0; i < tid; ++i) first &= sm.up[i] != up || sm.tok[i] != x;
      sm.rest[tid] = first ? to_mass(sm.px[tid]) : 0;
      const unsigned mask = __ballot_sync(0xffffffffu, first);
      if (lane == 0) sm.first[w] = mask;
    }
  }
  bad = __syncthreads_or(bad);
  if (!kDrawn && tid < kNodes) {
    Mass before = 0;
    for (int i = 0; i < tid; ++i) before += sm.up[i] == up ? sm.rest[i] : 0;
    const unsigned mask = __ballot_sync(0xffffffffu, up >= 0 && mass_times(less(kOne, before), sm.us[tid]) < sm.rest[tid]);
    if (lane == 0) sm.ok[w] = mask;
  }
  int* path = a.path + row * N;
  if (rank == 0 && tid == 0) a.token[row] = -1;  // (the clusters' barriers order it before the token itself)
  if (bad || sm.up[0] != -1) {
    if (rank == 0 && tid < N) path[tid] = -1;
    if (rank == 0 && tid == 0) {
      if (bad) atomicOr(&g_verify_error, 1u << 5);
      a.count[row] = 0;
    }
    if (C > 1) cluster_wait();
    return;
  }

  // this warp's run of the vocabulary
  int cur = 0;
  const int64_t runs = (int64_t)C * kVerifyWarps, len = ((V + runs - 1) / runs + 7) & ~(int64_t)7;
  auto run_at = [&](int64_t k, int off) { return k <= 0 ? 0 : k >= runs ? V : min(V, k * len - off); };
  int passes = 0;
  Mass total = 0, before = 0;  // of the last pass: of all, and of the CTAs before this one
  Mass* warp_sum = nullptr;    // and of this one's warps
  unsigned long long gone = 0;  // rejected children (drafts that were given), one per token
  bool waited = C == 1;
  auto place = [&](const T* P, const T* Q, int* off) {  // how the rows lie
    constexpr int n = Vec<T>::n;
    const uintptr_t p = reinterpret_cast<uintptr_t>(P), q = Q ? reinterpret_cast<uintptr_t>(Q) : p;
    *off = (int)(p / sizeof(T)) & (n - 1);
    return ((p ^ q) & 15u) == 0;
  };
  // the calling warp's sum over [lo, hi) of what is drawn from at the current node
  auto sum_of = [&](int64_t lo, int64_t hi, Mass S, bool plain) {
    const T* P = P0 + cur * V;
    const T* Q = plain || !kDrawn || S == 0 ? nullptr : Q0 + cur * V;
    int off;
    const bool vec = place(P, Q, &off);
    Mass sum = !kDrawn || !Q ? sum_run<T, kPlain>(P, Q, lo, hi, vec, off, S)
               : S == kOne   ? sum_first<T>(P, Q, lo, hi, vec, off)
                             : sum_run<T, kMore>(P, Q, lo, hi, vec, off, S);
    if (!kDrawn && !plain)
      for (unsigned long long g = gone; g; g &= g - 1) {
        const int i = __ffsll(g) - 1;
        if (sm.tok[i] >= lo && sm.tok[i] < hi) sum -= to_mass(sm.px[i]);
      }
    return sum;
  };
  auto pass = [&](Mass S, bool plain) {
    int off;
    place(P0 + cur * V, nullptr, &off);
    const int64_t k = (int64_t)rank * kVerifyWarps + w;
    const Mass sum = sum_of(run_at(k, off), run_at(k + 1, off), S, plain);
    warp_sum = sm.warp_sum[passes & 1];
    if (lane == 0) warp_sum[w] = sum;
    __syncthreads();
    Mass mine = 0;
    for (int i = 0; i < kVerifyWarps; ++i) mine += warp_sum[i];
    total = mine;
    before = 0;
    if (C > 1) {
      if (!waited) cluster_wait();  // all CTAs are there
      waited = true;
      Mass* slot = sm.cta_sum[passes & 1];
      if (tid < C) store_remote(slot + rank, tid, mine);
      __syncwarp();
      cluster_arrive();
      cluster_wait();
      total = 0;
      for (int i = 0; i < C; ++i) {
        if (i < rank) before += slot[i];
        total += slot[i];
      }
    }
    ++passes;
  };

  int count = 1, passed = -1;  // passed: the node of the last pass, with the present S
  if (rank == 0 && tid == 0) path[0] = 0;
  Mass S = 0, Z = kOne;
  const int up0 = sm.up[lane], up1 = sm.up[lane + 32];
  if (!kDrawn) __syncthreads();
  const unsigned long long ok_of = kDrawn ? 0 : sm.ok[0] | (unsigned long long)sm.ok[1] << 32;
  for (;;) {
    unsigned long long kids = __ballot_sync(0xffffffffu, up0 == cur) |
                              (unsigned long long)__ballot_sync(0xffffffffu, up1 == cur) << 32;
    int next = -1;
    if (!kDrawn) {
      if (kids & ok_of) next = __ffsll(kids & ok_of) - 1;
      else gone = kids & (sm.first[0] | (unsigned long long)sm.first[1] << 32);
    }
    for (; kDrawn && kids && next < 0; kids &= kids - 1) {
      const int i = __ffsll(kids) - 1;
      const float p = sm.px[i], u = sm.us[i], q = __saturatef(sm.qx[i]);
      bool ok;
      if (S == 0) {  // exactly: the product's rounding error decides where it is p
        const float t = u * q, e = fmaf(u, q, -t), sp = __saturatef(p);
        ok = t < sp || (t == sp && e < 0.f);
      } else {
        const Mass R = S == kOne ? rest_of<kFirst>(p, q, S) : rest_of<kMore>(p, q, S);
        ok = mass_times(mass_times(Z, q), u) < R;
      }
      if (ok) {
        next = i;
      } else {
        S += min(Z, kMost - S);
        pass(S, false);
        Z = total;
        passed = cur;
      }
    }
    if (next < 0) break;
    cur = next;
    S = 0;
    Z = kOne;
    passed = -1;
    if (rank == 0 && tid == 0) path[count] = cur;
    ++count;
  }
  if (rank == 0) {
    if (tid >= count && tid < N) path[tid] = -1;
    if (tid == 0) a.count[row] = count;
  }

  // the next token: the first index whose running sum passes u_0 of the whole
  bool plain = false;
  if (passed != cur) pass(S, false);
  if (total == 0) {  // nothing is left: from the target's row itself
    plain = true;
    pass(0, true);
  }
  if (total == 0) return;
  Mass target = min(mass_times(total, sm.us[0]), total - 1);
  Mass mine = 0;
  for (int i = 0; i < kVerifyWarps; ++i) mine += warp_sum[i];
  if (target < before || target - before >= mine) return;  // another CTA's
  target -= before;
  int run = 0;
  while (target >= warp_sum[run]) target -= warp_sum[run++];  // (ends: target is below their sum)
  const T* P = P0 + cur * V;
  const T* Q = plain || !kDrawn || S == 0 ? nullptr : Q0 + cur * V;
  int off;
  place(P, nullptr, &off);
  const int64_t k = (int64_t)rank * kVerifyWarps + run;
  int64_t lo = run_at(k, off), hi = run_at(k + 1, off);
  if (hi - lo > 4 * kVerifyThreads) {
    // an eighth of a long run per warp first, 16 bytes at a time: only the one that holds the token then goes to all
    // threads, whose few neighbouring values are read one by one (61 rows of 131072: 19.7 -> 15.1 us)
    const int64_t begin = lo, end = hi, len = ((hi - lo + kVerifyWarps - 1) / kVerifyWarps + 7) & ~(int64_t)7;
    auto part_at = [&](int i) { return i == 0 ? begin : i == kVerifyWarps ? end : min(end, begin + i * len - (begin ? 0 : off)); };
    const Mass part = sum_of(part_at(w), part_at(w + 1), S, plain);
    if (lane == 0) sm.part[w] = part;
    __syncthreads();
    int i = 0;
    while (target >= sm.part[i]) target -= sm.part[i++];  // (ends: they are the run's sum)
    lo = part_at(i);
    hi = part_at(i + 1);
  }
  const int64_t each = (hi - lo + kVerifyThreads - 1) / kVerifyThreads;
  const int64_t from = min(hi, lo + tid * each), to = min(hi, from + each);
  auto mass_at = [&](int64_t x) -> Mass {
    const float p = to_f32(P[x]);
    if (kDrawn && Q) return S == kOne ? rest_of<kFirst>(p, to_f32(Q[x]), S) : rest_of<kMore>(p, to_f32(Q[x]), S);
    if (!kDrawn && !plain)
      for (unsigned long long g = gone; g; g &= g - 1)
        if (sm.tok[__ffsll(g) - 1] == x) return 0;
    return to_mass(p);
  };
  Mass sum = 0;
#pragma unroll 4
  for (int64_t x = from; x < to; ++x) sum += mass_at(x);
  Mass upto = sum;  // over the threads up to this one
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Mass y = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += y;
  }
  if (lane == 31) sm.scan[w] = upto;
  __syncthreads();
  for (int i = 0; i < w; ++i) upto += sm.scan[i];
  if (upto - sum <= target && target < upto) {
    Mass cum = upto - sum;
    int64_t x = from;
    while (x < to - 1 && (cum += mass_at(x)) <= target) ++x;
    a.token[row] = (int)x;
  }
}

template <typename T>
cudaError_t launch(VerifyArgs a, int n, cudaStream_t s) {
  // CTAs per row: doubled while all of them run at once (four to an SM) and each has 2048 values
  a.split = 1;
  while (a.split < kVerifySplit && (int64_t)n * a.split * 2 <= 4 * sm_count() && a.V >= (int64_t)4096 * a.split) a.split *= 2;
  return launch_following(false, a.draft ? tree_verify_kernel<T, true> : tree_verify_kernel<T, false>, dim3((unsigned)n * a.split), kVerifyThreads, 0, a.split, s, a);
}

}  // namespace

cudaError_t launch_tree_verify(const int* parents, const int* tokens, const void* probs, const void* draft,
                               const float* u, int* path, int* count, int* token, int n, int N, int64_t V,
                               int dtype, cudaStream_t s) {
  VerifyArgs a;
  a.parents = parents; a.tokens = tokens; a.probs = probs; a.draft = draft; a.u = u; a.path = path;
  a.count = count; a.token = token; a.N = N; a.V = V; a.split = 1;
  return dtype == LL_F32 ? launch<float>(a, n, s) : launch<__nv_bfloat16>(a, n, s);
}

cudaError_t verify_take_error(cudaStream_t s, unsigned* flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_verify_error, sizeof(v), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && v) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbolAsync(g_verify_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  *flags = v;
  return e;
}

}  // namespace ll
