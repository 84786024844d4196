// Log-linear attention of a tree of drafted tokens over the paged decode cache.
//
// Node i of a row's tree, at depth d (a root: 0), stands at position t = pos + d behind the slot's
// pos positions and the nodes above it.  Its output is the decode step's, as if the path to it had
// been decoded:
//     out_i = sum over s <= t of lambda_i[level(t, s)] exp(log a behind s up to t) (q_i . k_s) v_s,
// s running over the context and the path.  Whole blocks come from the pages of block j = pos / 64:
// a node still in block j sees page m at level 7 + m, one in block j + 1 sees the pages below
// ctz(j + 1) and block j itself as one Fenwick bucket, level 7 + ctz(j + 1).  So a tree that
// runs over a block's end needs no fold, and nothing is written but the outputs.
#include "cache_common.cuh"

namespace ll {
namespace {

constexpr int kNodes = LL_TREE_MAX;

struct TreeArgs {
  const int* slots;
  const int* pos;
  const int* parents;
  const void* q;
  const void* k;
  const void* v;
  int64_t sq[3], sk[3], sv[3];  // elements from row to row, node to node, head to head
  const float* log_a;           // may be null
  const float* lam;
  void* out;
  int n, N, L;
};

constexpr int kTreeThreads = 256;

struct TreeSmem {
  float after[kW];                   // log decay from each token of the block to the context's last
  float first[kNodes];               // log decay of the path to each node
  float la[kNodes];
  float page_w[kMaxLevels][kNodes];  // weights of the live pages, lowest level first
  int page_at[kMaxLevels], page_lv[kMaxLevels];
  float page_log[kMaxLevels];
  int up[kNodes], depth[kNodes];
  unsigned long long above[kNodes];  // nodes on the path, itself included
  float since;
  unsigned bad;
};

// One CTA per (row, head).
template <typename T, typename OutT>
__global__ void __launch_bounds__(kTreeThreads) cache_tree_kernel(ll_cache c, TreeArgs a) {
  extern __shared__ __align__(16) float dyn[];  // q [N][dk], weights of tokens [N][64 + N]
  __shared__ TreeSmem sm;
  const int H = (int)c.H, G = (int)(c.H / c.Hqk), dk = (int)c.dk, dv = (int)c.dv, M = (int)c.levels;
  const int tid = threadIdx.x, lane = tid & 31, N = a.N;
  const int row = blockIdx.x / H, h = blockIdx.x - row * H;
  const int s = a.slots[row], pos = a.pos[row];
  if (s == -1) return;
  const unsigned why = row_bad(c, s, pos);
  if (why) {
    if (tid == 0 && h == 0) raise(c, why);
    return;
  }
  const int j = pos >> kLogW, r = pos & (kW - 1), par = j & 1, to = __ffs(j + 1) - 1, live = __popc(j);
  float* qs = dyn;
  float* ps = dyn + N * dk;
  const int width = kW + N;
  if (tid == 0) sm.bad = before_pages(c, s, pos) ? LL_CACHE_ERR_POSITION : 0;
  __syncthreads();
  if (tid < N) {
    const int up = a.parents[(int64_t)row * N + tid];
    const bool fine = up < tid && up >= -2;
    if (!fine) atomicOr(&sm.bad, LL_CACHE_ERR_TREE);
    sm.up[tid] = fine ? up : -2;
    sm.la[tid] = fine && up != -2 && a.log_a ? a.log_a[((int64_t)row * N + tid) * H + h] : 0.f;
  }
  if (tid >= kTreeThreads - 32) {
    const bool here = lane < M && (j >> lane) & 1;
    if (here) {
      const int at = __popc(j & ((1 << lane) - 1)), e = c.page_table[(int64_t)s * M + lane];
      sm.page_at[at] = e;
      sm.page_lv[at] = lane;
      sm.page_log[at] = c.page_log[(((int64_t)s * 2 + par) * M + lane) * H + h];
      if (e < 0 || e >= c.n_pages) atomicOr(&sm.bad, LL_CACHE_ERR_MISSING);
    }
  } else if (tid >= kTreeThreads - 64) {
    float since;
    block_decays(c.win_log_a + ((int64_t)s * H + h) * kW, r, c.page_from[s * 2 + par], sm.after, &since);
    if (lane == 0) sm.since = since;
  }
  const T* gq = static_cast<const T*>(a.q) + row * a.sq[0] + (h / G) * a.sq[2];
  const T* gk = static_cast<const T*>(a.k) + row * a.sk[0] + (h / G) * a.sk[2];
  const T* gv = static_cast<const T*>(a.v) + row * a.sv[0] + h * a.sv[2];
  for (int i = tid; i < N * dk; i += kTreeThreads) qs[i] = to_f32(gq[(i / dk) * a.sq[1] + i % dk]);
  __syncthreads();
  if (tid < N) {
    unsigned long long above = 0;
    int depth = -1;
    const bool in = sm.up[tid] != -2;
    for (int x = tid; in && x >= 0; x = sm.up[x]) {
      above |= 1ull << x;
      ++depth;
      if (sm.up[x] == -2) atomicOr(&sm.bad, LL_CACHE_ERR_TREE);  // a child of a node that is left out
    }
    if (in && !position_ok(c, (int64_t)pos + depth)) atomicOr(&sm.bad, LL_CACHE_ERR_POSITION);
    sm.above[tid] = above;
    sm.depth[tid] = depth;
  }
  __syncthreads();
  if (sm.bad) {
    if (tid == 0 && h == 0) raise(c, sm.bad);
    return;
  }
  if (tid < N && sm.up[tid] != -2) {
    const float* lam = a.lam + (((int64_t)row * N + tid) * H + h) * a.L;
    const int t = pos + sm.depth[tid];
    float acc = 0.f;  // log a behind x up to the node
    for (int x = tid; x >= 0; x = sm.up[x]) {
      ps[tid * width + kW + x] = lam[fenwick_level(t, pos + sm.depth[x])] * expf(acc);
      acc += sm.la[x];
    }
    sm.first[tid] = acc;
    for (int m = 0; m < live; ++m) {
      const int lv = (t >> kLogW) > j ? max(sm.page_lv[m], to) : sm.page_lv[m];
      sm.page_w[m][tid] = lam[kLogW + 1 + lv] * expf(sm.page_log[m] + sm.since + acc);
    }
  }
  __syncthreads();
  const T* wk = static_cast<const T*>(c.win_k) + ((int64_t)s * c.Hqk + h / G) * kW * dk;
  const T* wv = static_cast<const T*>(c.win_v) + ((int64_t)s * H + h) * kW * dv;
  for (int x = tid; x < N * width; x += kTreeThreads) {
    const int i = x / width, y = x - i * width;
    if (sm.up[i] == -2 || (y < kW ? y >= r : !(sm.above[i] >> (y - kW) & 1))) continue;
    const T* key = y < kW ? wk + y * dk : gk + (y - kW) * a.sk[1];
    float dot = 0.f;
    for (int d = 0; d < dk; ++d) dot = fmaf(qs[i * dk + d], to_f32(key[d]), dot);
    if (y < kW) {
      const float lam = a.lam[(((int64_t)row * N + i) * H + h) * a.L + fenwick_level(pos + sm.depth[i], (j << kLogW) + y)];
      ps[x] = lam * expf(sm.after[y] + sm.first[i]) * dot;
    } else {
      ps[x] *= dot;
    }
  }
  __syncthreads();
  // column `col` of nodes g, g + groups, ...
  const int groups = kTreeThreads / dv, col = tid % dv, g = tid / dv;
  if (g >= groups) return;
  float acc[kNodes / 2];
#pragma unroll
  for (int u = 0; u < kNodes / 2; ++u) acc[u] = 0.f;
  for (int y = 0; y < r; ++y) {
    const float x = to_f32(wv[y * dv + col]);
#pragma unroll
    for (int u = 0; u < kNodes / 2; ++u)
      if (g + u * groups < N) acc[u] = fmaf(ps[(g + u * groups) * width + y], x, acc[u]);
  }
  for (int y = 0; y < N; ++y) {
    const float x = to_f32(gv[y * a.sv[1] + col]);
#pragma unroll
    for (int u = 0; u < kNodes / 2; ++u)
      if (g + u * groups < N && sm.above[g + u * groups] >> y & 1)
        acc[u] = fmaf(ps[(g + u * groups) * width + kW + y], x, acc[u]);
  }
  for (int m = 0; m < live; ++m) {
    const float* P = c.pages + ((int64_t)sm.page_at[m] * H + h) * dk * dv + col;
    float part[kNodes / 2];
#pragma unroll
    for (int u = 0; u < kNodes / 2; ++u) part[u] = 0.f;
    for (int d = 0; d < dk; ++d) {
      const float x = P[d * dv];
#pragma unroll
      for (int u = 0; u < kNodes / 2; ++u)
        if (g + u * groups < N) part[u] = fmaf(qs[(g + u * groups) * dk + d], x, part[u]);
    }
#pragma unroll
    for (int u = 0; u < kNodes / 2; ++u)
      if (g + u * groups < N) acc[u] = fmaf(sm.page_w[m][g + u * groups], part[u], acc[u]);
  }
#pragma unroll
  for (int u = 0; u < kNodes / 2; ++u) {
    const int i = g + u * groups;
    if (i < N && sm.up[i] != -2)
      static_cast<OutT*>(a.out)[(((int64_t)row * N + i) * H + h) * dv + col] = from_f32<OutT>(acc[u]);
  }
}

template <typename T, typename OutT>
cudaError_t launch(const ll_cache& c, const TreeArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(float) * (size_t)a.N * (size_t)(c.dk + kW + a.N);
  const auto kernel = cache_tree_kernel<T, OutT>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)(a.n * c.H), kTreeThreads, smem, s>>>(c, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_tree(const ll_cache& c, const int* slots, const int* pos, const int* parents,
                              const void* q, const int64_t* sq, const void* k, const int64_t* sk,
                              const void* v, const int64_t* sv, const float* log_a, const float* lam,
                              void* out, int n, int N, int L, int out_dtype, cudaStream_t s) {
  TreeArgs a;
  a.slots = slots; a.pos = pos; a.parents = parents; a.q = q; a.k = k; a.v = v; a.log_a = log_a;
  a.lam = lam; a.out = out; a.n = n; a.N = N; a.L = L;
  for (int i = 0; i < 3; ++i) {
    a.sq[i] = sq[i];
    a.sk[i] = sk[i];
    a.sv[i] = sv[i];
  }
  const bool o32 = out_dtype == LL_F32;
  if (c.dtype == LL_F32) return o32 ? launch<float, float>(c, a, s) : launch<float, __nv_bfloat16>(c, a, s);
  return o32 ? launch<__nv_bfloat16, float>(c, a, s) : launch<__nv_bfloat16, __nv_bfloat16>(c, a, s);
}

}  // namespace ll
