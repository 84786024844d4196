// Appending accepted drafts to the paged decode cache: the nodes of a path join their slot as
// decode steps at pos, pos + 1, ... would have put them there, page reservation and fold included.
#include "cache_common.cuh"

namespace ll {
namespace {

struct AcceptArgs {
  const int* slots;
  const int* pos;
  const int* path;
  const void* k;
  const void* v;
  int64_t sk[3], sv[3];  // elements from row to row, node to node, head to head
  const float* log_a;    // may be null
  int* new_pos;
  int n, N, D;
};

// Nodes of the row's path (up to the first -1), or -1 where one of them is no node.
__device__ __forceinline__ int path_length(const AcceptArgs& a, int64_t row) {
  for (int d = 0; d < a.D; ++d) {
    const int x = a.path[row * a.D + d];
    if (x == -1) return d;
    if (x < 0 || x >= a.N) return -1;
  }
  return a.D;
}

// Why a row whose slot is in range cannot be served, before its pages are looked at.
__device__ __forceinline__ unsigned accept_bad(const ll_cache& c, int s, int pos, int count) {
  if (count < 0) return LL_CACHE_ERR_TREE;
  if (!position_ok(c, pos) || (count && !position_ok(c, (int64_t)pos + count - 1))) return LL_CACHE_ERR_POSITION;
  return before_pages(c, s, pos) ? LL_CACHE_ERR_POSITION : 0;
}

// As a reservation for each row's block: where the path ends the block, the page it is folded to.
// owner: the rows that are served, ~row of those that are left out.
__global__ void __launch_bounds__(kPlanThreads) accept_plan_kernel(ll_cache c, AcceptArgs a) {
  __shared__ int slot_s[kPlanThreads], block_s[kPlanThreads], count_s[kPlanThreads];
  const Scratch sc = scratch_of(c);
  const int tid = threadIdx.x, lane = tid & 31;
  let_next_start();
  const bool few = a.n <= kPlanThreads;
  if (few) {
    const int s = tid < a.n ? a.slots[tid] : -1, pos = tid < a.n ? a.pos[tid] : 0;
    slot_s[tid] = s;
    for (int r = tid >> 5; r < a.n; r += kPlanThreads / 32) {  // a warp per path
      const int x = lane < a.D ? a.path[(int64_t)r * a.D + lane] : -1;
      const int y = lane + 32 < a.D ? a.path[(int64_t)r * a.D + lane + 32] : -1;
      const unsigned end0 = __ballot_sync(0xffffffffu, x < 0 || x >= a.N), end1 = __ballot_sync(0xffffffffu, y < 0 || y >= a.N);
      const int len = end0 ? __ffs(end0) - 1 : end1 ? 31 + __ffs(end1) : 64;
      const int z = len < 32 ? __shfl_sync(0xffffffffu, x, len & 31) : __shfl_sync(0xffffffffu, y, len & 31);
      if (lane == 0) count_s[r] = len < 64 && z != -1 ? -1 : len;
    }
    __syncthreads();
    bool bad = s < -1 || s >= c.slots;
    if (s >= 0)
      for (int i = 0; i < tid; ++i) bad |= slot_s[i] == s;
    if (bad) raise(c, LL_CACHE_ERR_SLOT);
    const bool named = s >= 0 && !bad;
    const int count = tid < a.n ? count_s[tid] : 0;
    const unsigned why = named ? accept_bad(c, s, pos, count) : 0;
    if (why) raise(c, why);
    if (named) sc.owner[s] = why ? ~tid : tid;
    __syncthreads();
    slot_s[tid] = named && !why ? s : -1;
    block_s[tid] = pos >> kLogW;
    count_s[tid] = (pos & (kW - 1)) + count >= kW;
    __syncthreads();
    settle_pages(c, a.n, [&](int64_t r) { return slot_s[r]; }, [&](int64_t r) { return block_s[r]; },
                 [&](int64_t r) { return count_s[r] != 0; });
    return;
  }
  claim_slots(c, a.slots, a.n, sc.owner);
  __syncthreads();
  for (int64_t r = tid; r < a.n; r += kPlanThreads) {
    const int s = a.slots[r];
    if (!owns(c, sc.owner, s, r)) continue;
    const unsigned why = accept_bad(c, s, a.pos[r], path_length(a, r));
    if (why) raise(c, why);
    if (why) sc.owner[s] = ~(int)r;
  }
  __syncthreads();
  settle_pages(c, a.n, [&](int64_t r) { return owns(c, sc.owner, a.slots[r], r) ? a.slots[r] : -1; },
               [&](int64_t r) { return a.pos[r] >> kLogW; },
               [&](int64_t r) { return (a.pos[r] & (kW - 1)) + path_length(a, r) >= kW; });
}

constexpr int kAcceptThreads = 256;

// A row's fold, as far as its CTAs have to agree on it.
struct Fold {
  int dest;      // the page, -1 without a fold
  unsigned why;  // the row cannot be served
};
__device__ __forceinline__ Fold fold_of(const ll_cache& c, int s, int pos, int count) {
  Fold f = {-1, 0};
  const int j = pos >> kLogW, M = (int)c.levels, to = __ffs(j + 1) - 1;
  if ((pos & (kW - 1)) + count < kW) return f;
  for (int m = 0; m < M; ++m) {
    if (m != to && !(j >> m & 1)) continue;
    const int e = c.page_table[(int64_t)s * M + m];
    if (e < 0 || e >= c.n_pages || (m == to && c.refcount[e] != 1)) f.why = LL_CACHE_ERR_MISSING;
    else if (m == to) f.dest = e;
  }
  return f;
}

// One CTA per (row, head): the block that ends with the path, folded.
template <typename T>
__global__ void __launch_bounds__(kAcceptThreads) accept_fold_kernel(ll_cache c, AcceptArgs a) {
  __shared__ float tok[kW], since_s;
  const int H = (int)c.H, G = (int)(c.H / c.Hqk), dk = (int)c.dk, dv = (int)c.dv, M = (int)c.levels;
  const int tid = threadIdx.x, row = blockIdx.x / H, h = blockIdx.x - row * H, s = a.slots[row], pos = a.pos[row];
  wait_for_previous();
  if (!owns(c, scratch_of(c).owner, s, row)) return;
  const int count = path_length(a, row), j = pos >> kLogW, r = pos & (kW - 1), par = j & 1, to = __ffs(j + 1) - 1;
  const Fold f = fold_of(c, s, pos, count);
  if (f.why && tid == 0 && h == 0) raise(c, f.why);
  if (f.why || f.dest < 0) return;
  const int* path = a.path + (int64_t)row * a.D;
  if (tid < 32) {
    auto la = [&](int i) {
      if (i < r) return c.win_log_a[((int64_t)s * H + h) * kW + i];
      return a.log_a ? a.log_a[((int64_t)row * a.N + path[i - r]) * H + h] : 0.f;
    };
    float since;
    block_decays(la(tid), la(tid + 32), kW, c.page_from[s * 2 + par], tok, &since);
    tok[tid] = expf(tok[tid]);
    tok[tid + 32] = expf(tok[tid + 32]);
    since_s = since;
  }
  __syncthreads();
  const T* wk = static_cast<const T*>(c.win_k) + ((int64_t)s * c.Hqk + h / G) * kW * dk;
  const T* wv = static_cast<const T*>(c.win_v) + ((int64_t)s * H + h) * kW * dv;
  const T* gk = static_cast<const T*>(a.k) + row * a.sk[0] + (h / G) * a.sk[2];
  const T* gv = static_cast<const T*>(a.v) + row * a.sv[0] + h * a.sv[2];
  float* D = c.pages + ((int64_t)f.dest * H + h) * dk * dv;
  for (int x = tid; x < dk * dv; x += kAcceptThreads) {
    const int d = x / dv, e = x - d * dv;
    float sum = 0.f;
    for (int m = 0; m < to; ++m) {
      const float w = expf(c.page_log[(((int64_t)s * 2 + par) * M + m) * H + h] + since_s);
      sum = fmaf(w, c.pages[((int64_t)c.page_table[(int64_t)s * M + m] * H + h) * dk * dv + x], sum);
    }
    for (int i = 0; i < kW; ++i) {
      const float key = to_f32(i < r ? wk[i * dk + d] : gk[path[i - r] * a.sk[1] + d]);
      sum = fmaf(tok[i] * key, to_f32(i < r ? wv[i * dv + e] : gv[path[i - r] * a.sv[1] + e]), sum);
    }
    D[x] = sum;
  }
  // what the next block's calls read
  for (int m = tid; m < M; m += kAcceptThreads)
    if (m == to) c.page_log[(((int64_t)s * 2 + 1 - par) * M + m) * H + h] = 0.f;
    else if (m > to && (j >> m & 1))
      c.page_log[(((int64_t)s * 2 + 1 - par) * M + m) * H + h] = c.page_log[(((int64_t)s * 2 + par) * M + m) * H + h] + since_s;
  if (h == 0 && tid == 0) c.page_from[s * 2 + 1 - par] = 0;
}

// One CTA per (row, head): the path's tokens to their places.
template <typename T>
__global__ void __launch_bounds__(kAcceptThreads) accept_tokens_kernel(ll_cache c, AcceptArgs a) {
  const int H = (int)c.H, G = (int)(c.H / c.Hqk), dk = (int)c.dk, dv = (int)c.dv;
  const int tid = threadIdx.x, row = blockIdx.x / H, h = blockIdx.x - row * H, s = a.slots[row], pos = a.pos[row];
  if (!owns(c, scratch_of(c).owner, s, row)) return;
  const int count = path_length(a, row);
  if (fold_of(c, s, pos, count).why) return;
  const T* gk = static_cast<const T*>(a.k) + row * a.sk[0] + (h / G) * a.sk[2];
  const T* gv = static_cast<const T*>(a.v) + row * a.sv[0] + h * a.sv[2];
  for (int d = 0; d < count; ++d) {
    const int x = a.path[(int64_t)row * a.D + d], i = (pos + d) & (kW - 1);
    if (h % G == 0)
      for (int e = tid; e < dk; e += kAcceptThreads)
        static_cast<T*>(c.win_k)[(((int64_t)s * c.Hqk + h / G) * kW + i) * dk + e] = gk[x * a.sk[1] + e];
    for (int e = tid; e < dv; e += kAcceptThreads)
      static_cast<T*>(c.win_v)[(((int64_t)s * H + h) * kW + i) * dv + e] = gv[x * a.sv[1] + e];
    if (tid == 0)
      c.win_log_a[((int64_t)s * H + h) * kW + i] = a.log_a ? a.log_a[((int64_t)row * a.N + x) * H + h] : 0.f;
  }
  if (h == 0 && tid == 0) a.new_pos[row] = pos + count;
}

template <typename T>
cudaError_t launch(const ll_cache& c, const AcceptArgs& a, cudaStream_t s) {
  accept_plan_kernel<<<1, kPlanThreads, 0, s>>>(c, a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(a.n * c.H);
  e = launch_following(true, accept_fold_kernel<T>, dim3(grid), kAcceptThreads, 0, 1, s, c, a);
  if (e != cudaSuccess) return e;
  accept_tokens_kernel<T><<<grid, kAcceptThreads, 0, s>>>(c, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_accept(const ll_cache& c, const int* slots, const int* pos, const int* path,
                                const void* k, const int64_t* sk, const void* v, const int64_t* sv,
                                const float* log_a, int* new_pos, int n, int N, int D, cudaStream_t s) {
  AcceptArgs a;
  a.slots = slots; a.pos = pos; a.path = path; a.k = k; a.v = v; a.log_a = log_a; a.new_pos = new_pos;
  a.n = n; a.N = N; a.D = D;
  for (int i = 0; i < 3; ++i) {
    a.sk[i] = sk[i];
    a.sv[i] = sv[i];
  }
  return c.dtype == LL_F32 ? launch<float>(c, a, s) : launch<__nv_bfloat16>(c, a, s);
}

}  // namespace ll
