// Verification of a tree of drafted tokens against the target's probabilities (speculative
// sampling), from given random numbers.
//
// The walk starts at node 0, the pending token, and tries the current node's children in the order of their
// index, against what is left of the target's distribution P there: R_0 = P, Z_0 = 1.  A child with
// token x and random number u is accepted where
//     u Z_k < R_k(x)              (drafts that were given: x is removed from R when it is rejected)
//     u Z_k q(x) < R_k(x)         (drafts drawn from q: then R_{k+1} = max(R_k - Z_k q, 0), Z_{k+1} = sum of it)
// and else the next one is tried; where none is left the next token is drawn from R_k.  So the
// tokens are distributed as the target's own.  R_k is max(P - S_k q, 0) with S_k = Z_0 + .. + Z_{k-1}, as
// what has once reached 0 stays there: one multiply-add per value, whatever was rejected before.
//
// Sums over a vocabulary are 64-bit fixed point with 52 fractional bits: exact for values of
// 2^-28 and above, cut at 2^-52 below, and the same in every order, so the token drawn depends on
// no launch shape (fp32 sums move the boundaries of 1e5 tokens by more than the tokens' own
// width; fp64 adds run at 1/64 of the rate).
#include "ll_internal.cuh"

namespace ll {
namespace {

__device__ unsigned g_verify_error;

constexpr int kNodes = LL_TREE_MAX;
constexpr int kFraction = 52;
typedef unsigned long long Mass;

// x as fixed point; below 0 and NaN: 0, above 1: 1.
__device__ __forceinline__ Mass to_mass(float x) {
  const unsigned b = __float_as_uint(__saturatef(x));
  const Mass m = (Mass)(b & 0x7fffffu | 0x800000u) << (kFraction - 23);  // of an x in [1, 2)
  return m >> min(127u - (b >> 23), 63u);
}
// floor(s x) for x in [0, 1], s < 2^62.
__device__ __forceinline__ Mass mass_times(Mass s, float x) {
  const unsigned b = __float_as_uint(__saturatef(x)), m = b & 0x7fffffu | 0x800000u;
  const Mass lo = (s & 0xffffffffu) * m, hi = (s >> 32) * m + (lo >> 32);  // s m = hi 2^32 + low word of lo
  // s m 2^-23 2^-(127 - exponent)
  const unsigned shift = 127u - (b >> 23);
  const Mass x23 = hi << 9 | (lo & 0xffffffffu) >> 23;
  return x23 >> min(shift, 63u);
}

struct VerifyArgs {
  const int* parents;
  const int* tokens;
  const void* probs;
  const void* draft;  // may be null
  const float* u;
  int* path;
  int* count;
  int* token;
  int n, N;
  int64_t V;
};

constexpr int kVerifyThreads = 512;

__device__ Mass block_sum(Mass x, Mass* part) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  Mass t = 0;
  for (int i = 0; i < kVerifyThreads / 32; ++i) t += part[i];
  return t;
}

// One CTA per row.
template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) tree_verify_kernel(VerifyArgs a) {
  __shared__ int up[kNodes], tok[kNodes];
  __shared__ float px[kNodes], qx[kNodes], us[kNodes];
  __shared__ Mass part[kVerifyThreads / 32];
  __shared__ unsigned bad_s;
  __shared__ int hit;
  const int tid = threadIdx.x, N = a.N, row = blockIdx.x;
  const int64_t V = a.V;
  if (tid == 0) {
    bad_s = 0;
    hit = kNodes;
  }
  __syncthreads();
  const T* P0 = static_cast<const T*>(a.probs) + (int64_t)row * N * V;
  const T* Q0 = a.draft ? static_cast<const T*>(a.draft) + (int64_t)row * N * V : nullptr;
  if (tid < N) {
    const int p = a.parents[(int64_t)row * N + tid], x = a.tokens[(int64_t)row * N + tid];
    const bool child = p >= 0 && p < tid;
    const bool fine = child ? x >= 0 && x < V : p == -1 || p == -2;
    if (!fine) bad_s = 1;
    up[tid] = child && fine ? p : p == -1 ? -1 : -2;
    tok[tid] = x;
    px[tid] = child && fine ? to_f32(P0[p * V + x]) : 0.f;
    qx[tid] = child && fine && Q0 ? to_f32(Q0[p * V + x]) : 0.f;
    us[tid] = fminf(fmaxf(a.u[(int64_t)row * N + tid], 0.f), 0x1.fffffep-1f);
  }
  __syncthreads();
  if (tid < N && up[tid] >= 0 && up[up[tid]] == -2) bad_s = 1;
  __syncthreads();
  int* path = a.path + (int64_t)row * N;
  for (int i = tid; i < N; i += kVerifyThreads) path[i] = -1;
  if (bad_s || up[0] != -1) {
    if (tid == 0) {
      if (bad_s) atomicOr(&g_verify_error, 1u << 5);
      a.count[row] = 0;
      a.token[row] = -1;
    }
    return;
  }
  __syncthreads();
  int cur = 0, count = 1;
  if (tid == 0) path[0] = 0;
  const Mass one = 1ull << kFraction;
  Mass S = 0, Z = one;
  unsigned long long gone = 0;  // rejected children (drafts that were given)
  for (int i = 1; i < N; ++i) {
    if (up[i] != cur) continue;
    bool ok;
    const double z = (double)Z * 0x1p-52 * (double)us[i];
    if (!Q0) {
      bool left = true;
      for (int x = cur + 1; x < i; ++x) left &= !(gone >> x & 1) || tok[x] != tok[i];
      const Mass R = left ? to_mass(px[i]) : 0;
      ok = z < (double)R * 0x1p-52;
      if (!ok) {
        Z -= R < Z ? R : Z;
        gone |= 1ull << i;
      }
    } else {
      const Mass p = to_mass(px[i]), q = mass_times(S, qx[i]);
      ok = z * (double)__saturatef(qx[i]) < (double)(p > q ? p - q : 0) * 0x1p-52;
      if (!ok) {
        S += Z;
        Mass sum = 0;
        for (int64_t x = tid; x < V; x += kVerifyThreads) {
          const Mass p1 = to_mass(to_f32(P0[cur * V + x])), q1 = mass_times(S, to_f32(Q0[cur * V + x]));
          sum += p1 > q1 ? p1 - q1 : 0;
        }
        Z = block_sum(sum, part);
      }
    }
    if (ok) {
      cur = i;
      S = 0;
      Z = one;
      gone = 0;
      if (tid == 0) path[count] = i;
      ++count;
    }
  }
  // the next token: the first index whose running sum passes u_0 of the whole
  auto mass_of = [&](int64_t x, bool full) -> Mass {
    const Mass p = to_mass(to_f32(P0[cur * V + x]));
    if (full) return p;
    if (Q0) {
      const Mass q = S ? mass_times(S, to_f32(Q0[cur * V + x])) : 0;
      return p > q ? p - q : 0;
    }
    for (unsigned long long g = gone; g; g &= g - 1)
      if (tok[__ffsll(g) - 1] == x) return 0;
    return p;
  };
  const int64_t share = (V + kVerifyThreads - 1) / kVerifyThreads, lo = min(V, tid * share), hi = min(V, lo + share);
  for (int full = 0; full < 2; ++full) {
    Mass sum = 0;
    for (int64_t x = lo; x < hi; ++x) sum += mass_of(x, full);
    const Mass total = block_sum(sum, part);
    if (total == 0) continue;  // nothing is left: from the target's row itself
    Mass before = sum;  // over the threads before this one
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Mass y = __shfl_up_sync(0xffffffffu, before, d);
      if ((tid & 31) >= d) before += y;
    }
    before -= sum;
    for (int i = 0; i < tid >> 5; ++i) before += part[i];
    const Mass target = mass_times(total, us[0]);
    if (before <= target && target < before + sum) {
      int64_t x = lo;
      for (Mass cum = before; x < hi; ++x)
        if ((cum += mass_of(x, full)) > target) break;
      a.token[row] = (int)x;
      hit = 1;
    }
    break;
  }
  __syncthreads();
  if (tid == 0) {
    a.count[row] = count;
    if (hit != 1) a.token[row] = -1;
  }
}

}  // namespace

cudaError_t launch_tree_verify(const int* parents, const int* tokens, const void* probs, const void* draft,
                               const float* u, int* path, int* count, int* token, int n, int N, int64_t V,
                               int dtype, cudaStream_t s) {
  VerifyArgs a;
  a.parents = parents; a.tokens = tokens; a.probs = probs; a.draft = draft; a.u = u; a.path = path;
  a.count = count; a.token = token; a.n = n; a.N = N; a.V = V;
  if (dtype == LL_F32) tree_verify_kernel<float><<<n, kVerifyThreads, 0, s>>>(a);
  else tree_verify_kernel<__nv_bfloat16><<<n, kVerifyThreads, 0, s>>>(a);
  return cudaGetLastError();
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
