// Appending accepted drafts to the paged decode cache: the nodes of a path join their slot as
// decode steps at pos, pos + 1, ... would have put them there, page reservation and fold included.
//
// Two kernels: a plan in one CTA, which claims the slots and settles the pages (3 us, twice that where blocks end), and a
// CTA per (row, head), launched while the plan runs.  Measured (GB300, calls in a row; floor: bytes at the measured
// copy rate): one sequence's path 5.6 us; 125 rows of 16 heads, d 128, ten of which end a block, 39 us (floor
// 5.7): 13 without the ten, 24 with those that fold to no older page, and the rest is the one that folds seven pages, by
// one CTA per head at 30 GB/s each; 32 rows of 48 heads, dv 64, all of which end a block: 45 us, 109 MB, floor 16.
// Folds on the CUDA cores: those of fp32 tokens 214 us (batch: 83), 123 MB, floor 18, bound by the latency of their reads
// with two CTAs per SM (25 % of the issue slots); bf16 of d_k 72 and d_v 36 130 us, 38 MB, floor 6.
// CTAs of 128 (53, 46 us) or 512 threads (39, 62), persistent ones with a list of folds (36 to 48, 69 and more), and
// pages through a ring in shared memory (47, 53) were no better.
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
__device__ __forceinline__ unsigned accept_bad(const ll_cache& c, int pos, int count, bool before) {
  if (count < 0) return LL_CACHE_ERR_TREE;
  if (!position_ok(c, pos) || (count && !position_ok(c, (int64_t)pos + count - 1))) return LL_CACHE_ERR_POSITION;
  return before ? LL_CACHE_ERR_POSITION : 0;
}

// As a reservation for each row's block: where the path ends the block, the page it is folded to.
// owner: the rows that are served, ~row of those that are left out.
__global__ void __launch_bounds__(kPlanThreads) accept_plan_kernel(ll_cache c, AcceptArgs a) {
  __shared__ int slot_s[kPlanThreads], count_s[kPlanThreads];
  const Scratch sc = scratch_of(c);
  const int tid = threadIdx.x, lane = tid & 31;
  let_next_start();
  if (a.n <= kPlanThreads) {  // a row per thread
    const int s = tid < a.n ? a.slots[tid] : -1, pos = tid < a.n ? a.pos[tid] : 0;
    slot_s[tid] = s;
    // what may be needed, ahead of knowing (the last block has no page to be folded to)
    bool bad = s < -1 || s >= c.slots, shared = false, before = false;
    int e = -1;
    if (s >= 0 && !bad && position_ok(c, pos)) {
      before = before_pages(c, s, pos);
      if ((pos >> kLogW) + 1 < 1 << c.levels) e = fold_page(c, s, pos >> kLogW, &shared);
    }
    for (int r = tid >> 5; r < a.n; r += kPlanThreads / 32) {  // a warp per path
      const int x = lane < a.D ? a.path[(int64_t)r * a.D + lane] : -1;
      const int y = lane + 32 < a.D ? a.path[(int64_t)r * a.D + lane + 32] : -1;
      const unsigned end0 = __ballot_sync(0xffffffffu, x < 0 || x >= a.N), end1 = __ballot_sync(0xffffffffu, y < 0 || y >= a.N);
      const int len = end0 ? __ffs(end0) - 1 : end1 ? 31 + __ffs(end1) : 64;
      const int z = len < 32 ? __shfl_sync(0xffffffffu, x, len & 31) : __shfl_sync(0xffffffffu, y, len & 31);
      if (lane == 0) count_s[r] = len < 64 && z != -1 ? -1 : len;
    }
    __syncthreads();
    if (s >= 0)
      for (int i = 0; i < tid; ++i) bad |= slot_s[i] == s;
    if (bad) raise(c, LL_CACHE_ERR_SLOT);
    const bool named = s >= 0 && !bad;
    const int count = tid < a.n ? count_s[tid] : 0;
    const unsigned why = named ? accept_bad(c, pos, count, before) : 0;
    if (why) raise(c, why);
    if (named) {
      sc.owner[s] = why ? ~tid : tid;
      sc.done[s] = 0;
    }
    settle_few(c, a.n, named && !why ? s : -1, pos >> kLogW, (pos & (kW - 1)) + count >= kW, e, shared);
    return;
  }
  claim_slots(c, a.slots, a.n, sc.owner);
  __syncthreads();
  for (int64_t r = tid; r < a.n; r += kPlanThreads) {
    const int s = a.slots[r];
    if (!owns(c, sc.owner, s, r)) continue;
    const int pos = a.pos[r];
    const unsigned why = accept_bad(c, pos, path_length(a, r), position_ok(c, pos) && before_pages(c, s, pos));
    if (why) raise(c, why);
    if (why) sc.owner[s] = ~(int)r;
    sc.done[s] = 0;
  }
  __syncthreads();
  settle_pages(c, a.n, [&](int64_t r) { return owns(c, sc.owner, a.slots[r], r) ? a.slots[r] : -1; },
               [&](int64_t r) { return a.pos[r] >> kLogW; },
               [&](int64_t r) { return (a.pos[r] & (kW - 1)) + path_length(a, r) >= kW; });
}

constexpr int kAcceptThreads = 256, kAcceptWarps = kAcceptThreads / 32;
constexpr int kTogether = 2;  // pages whose loads are on their way together, 8 of a thread
constexpr int kPad = 8;  // elements that set a token's row off by 16 bytes

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}

// Rows of `width` elements from src_of(row) to dst_of(row), by the CTA; whole 16-byte pieces (vec), four of a thread
// on their way, or elements.
template <typename T, typename Src, typename Dst>
__device__ __forceinline__ void copy_tokens(int rows, int width, bool vec, Src src_of, Dst dst_of) {
  constexpr int per = 16 / sizeof(T), kLanes = 128 / per, kStep = kAcceptThreads / kLanes;  // pieces of 128 columns
  if (vec) {
    const int x = (threadIdx.x & (kLanes - 1)) * per;
    if (x < width)
      for (int r0 = threadIdx.x / kLanes; r0 < rows; r0 += 4 * kStep) {
        uint4 y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (r0 + u * kStep < rows) y[u] = *reinterpret_cast<const uint4*>(src_of(r0 + u * kStep) + x);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (r0 + u * kStep < rows) *reinterpret_cast<uint4*>(dst_of(r0 + u * kStep) + x) = y[u];
      }
  } else {
    const int x = threadIdx.x & 127;
    if (x < width)
      for (int r = threadIdx.x >> 7; r < rows; r += kAcceptThreads >> 7) dst_of(r)[x] = src_of(r)[x];
  }
}

constexpr int kTokenHeads = 4;  // heads of a CTA that only copies tokens

// Tokens d0 .. d1 - 1 of the row's path, the first of which follows r tokens of the block (they stay inside one),
// to their places: the values of heads [h0, h1), the keys [q0, q1).
template <typename T>
__device__ __forceinline__ void put_values(const ll_cache& c, const AcceptArgs& a, int row, int s, int r, const int* path,
                                           int d0, int d1, int h0, int h1) {
  const int H = (int)c.H, dv = (int)c.dv, n = d1 - d0, at = (r + d0) & (kW - 1);
  const T* gv = static_cast<const T*>(a.v) + row * a.sv[0];
  T* wv = static_cast<T*>(c.win_v) + ((int64_t)s * H * kW + at) * dv;
  const bool vec = ((dv | a.sv[0] | a.sv[1] | a.sv[2]) * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(a.v) & 15u) == 0;
  copy_tokens<T>(n * (h1 - h0), dv, vec, [&](int i) { return gv + (h0 + i / n) * a.sv[2] + path[d0 + i % n] * a.sv[1]; },
                 [&](int i) { return wv + (int64_t)((h0 + i / n) * kW + i % n) * dv; });
  for (int i = threadIdx.x; i < n * (h1 - h0); i += kAcceptThreads) {
    const int h = h0 + i / n, d = i % n;
    c.win_log_a[((int64_t)s * H + h) * kW + at + d] = a.log_a ? a.log_a[((int64_t)row * a.N + path[d0 + d]) * H + h] : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void put_keys(const ll_cache& c, const AcceptArgs& a, int row, int s, int r, const int* path, int d0,
                                         int d1, int q0, int q1) {
  const int dk = (int)c.dk, n = d1 - d0, at = (r + d0) & (kW - 1);
  const T* gk = static_cast<const T*>(a.k) + row * a.sk[0];
  T* wk = static_cast<T*>(c.win_k) + ((int64_t)s * c.Hqk * kW + at) * dk;
  const bool vec = ((dk | a.sk[0] | a.sk[1] | a.sk[2]) * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(a.k) & 15u) == 0;
  copy_tokens<T>(n * (q1 - q0), dk, vec, [&](int i) { return gk + (q0 + i / n) * a.sk[2] + path[d0 + i % n] * a.sk[1]; },
                 [&](int i) { return wk + (int64_t)((q0 + i / n) * kW + i % n) * dk; });
}

// One CTA per (row, head): the path's tokens to their places and, where they end the block, its fold: the sum
// of the pages below the level that it goes to, decayed, and of the 64 tokens' products.  kMma: bf16 tokens of whole
// 16-byte pieces, whose products run on the tensor cores, exact keys against decayed values in three bf16
// parts, as in the step; else fp32 multiply-adds.  Tokens of the next block replace those that the fold reads: a head's own
// values behind its own reads, the keys that heads share by the row's last CTA to have read them.
template <typename T, bool kMma>
__global__ void __launch_bounds__(kAcceptThreads, kMma ? 4 : 2) accept_kernel(ll_cache c, AcceptArgs a) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ __align__(8) float tok[kW];
  __shared__ float page_e[kMaxLevels];
  __shared__ int page_at[kMaxLevels], path[LL_TREE_MAX];
  __shared__ int count_s, last_s;
  __shared__ unsigned why_s;
  const int H = (int)c.H, Hqk = (int)c.Hqk, G = H / Hqk, dk = (int)c.dk, dv = (int)c.dv, M = (int)c.levels;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int row = blockIdx.x / H, h = blockIdx.x - row * H, hq = h / G;
  const int s = a.slots[row], pos = a.pos[row];
  const int j = pos >> kLogW, r = pos & (kW - 1), par = j & 1, to = __ffs(j + 1) - 1;
  if (w == 0) {
    const int x = lane < a.D ? a.path[(int64_t)row * a.D + lane] : -1, y = lane + 32 < a.D ? a.path[(int64_t)row * a.D + lane + 32] : -1;
    path[lane] = x;
    path[lane + 32] = y;
    const unsigned x_end = __ballot_sync(0xffffffffu, x < 0), y_end = __ballot_sync(0xffffffffu, y < 0);
    if (lane == 0) count_s = x_end ? __ffs(x_end) - 1 : y_end ? 31 + __ffs(y_end) : 64;
  }
  wait_for_previous();  // what the plan has settled
  const Scratch sc = scratch_of(c);
  const bool served = owns(c, sc.owner, s, row);
  if (w == 1) {  // the fold's pages, in case (where there is one to go to, the plan has made it the slot's own)
    const bool here = served && lane < M && (lane == to || (j >> lane & 1));
    const int e = here ? c.page_table[(int64_t)s * M + lane] : 0;
    if (lane < M) page_at[lane] = e;
    const bool why = __any_sync(0xffffffffu, e < 0 || e >= c.n_pages);
    if (lane == 0) why_s = why ? LL_CACHE_ERR_MISSING : 0;
  }
  __syncthreads();
  if (!served) return;
  const int count = count_s;
  const bool fold = r + count >= kW;
  if (fold && why_s) {
    if (tid == 0 && h == 0) raise(c, why_s);
    return;
  }
  if (!fold) {  // a few heads by one CTA
    const int h1 = min(H, h + kTokenHeads);
    if (h % kTokenHeads) return;
    put_values<T>(c, a, row, s, r, path, 0, count, h, h1);
    put_keys<T>(c, a, row, s, r, path, 0, count, (h + G - 1) / G, (h1 + G - 1) / G);  // whose first head is among them
    if (h == 0 && tid == 0) a.new_pos[row] = pos + count;
    return;
  }
  const T* gk = static_cast<const T*>(a.k) + row * a.sk[0] + hq * a.sk[2];
  const T* gv = static_cast<const T*>(a.v) + row * a.sv[0] + h * a.sv[2];
  const float* ga = a.log_a ? a.log_a + (int64_t)row * a.N * H + h : nullptr;
  const T* wk = static_cast<const T*>(c.win_k) + ((int64_t)s * Hqk + hq) * kW * dk;
  const T* wv = static_cast<const T*>(c.win_v) + ((int64_t)s * H + h) * kW * dv;
  const float* wa = c.win_log_a + ((int64_t)s * H + h) * kW;
  const int ends = kW - r;  // tokens of the path in this block
  // the 64 tokens, of the block and of the path
  auto key = [&](int i) { return i < r ? wk + i * dk : gk + path[i - r] * a.sk[1]; };
  auto value = [&](int i) { return i < r ? wv + i * dv : gv + path[i - r] * a.sv[1]; };
  const int kp = kMma ? dk + kPad : (dk + 3) & ~3, vp = kMma ? dv + kPad : dv;
  __nv_bfloat16* ks = reinterpret_cast<__nv_bfloat16*>(dyn);
  __nv_bfloat16* vs = ks + kW * kp;
  float* kf = reinterpret_cast<float*>(dyn);
  float* vf = kf + kW * kp;
  if constexpr (kMma) {
    const int x = (tid & 15) * 8;
    for (int i = tid >> 4; i < kW; i += kAcceptThreads / 16) {
      if (x < dk) cp_async16(ks + i * kp + x, key(i) + x);
      if (x < dv) cp_async16(vs + i * vp + x, value(i) + x);
    }
  } else {
    const int x = tid & 127;
#pragma unroll 4
    for (int i = tid >> 7; i < kW; i += kAcceptThreads >> 7) {
      if (x < kp) kf[i * kp + x] = x < dk ? to_f32(key(i)[x]) : 0.f;
      if (x < dv) vf[i * vp + x] = to_f32(value(i)[x]);
    }
  }
  if (w == 0) {
    auto la = [&](int i) { return i < r ? wa[i] : ga ? ga[(int64_t)path[i - r] * H] : 0.f; };
    float since;
    block_decays(la(lane), la(lane + 32), kW, c.page_from[s * 2 + par], tok, &since);
    tok[lane] = expf(tok[lane]);
    tok[lane + 32] = expf(tok[lane + 32]);
    const bool here = lane < M && (j >> lane & 1);
    float* log = c.page_log + ((int64_t)s * 2 * M + lane) * H + h;
    const float old = here ? log[(int64_t)par * M * H] + since : 0.f;
    if (here && lane < to) page_e[lane] = expf(old);
    // what the next block's calls read
    if (lane < M && (lane == to || (here && lane > to))) log[(int64_t)(1 - par) * M * H] = lane == to ? 0.f : old;
    if (h == 0 && lane == 0) c.page_from[s * 2 + 1 - par] = 0;
  }
  __syncthreads();
  const int64_t size = (int64_t)dk * dv;
  float* D = c.pages + ((int64_t)page_at[to] * H + h) * size;
  auto page = [&](int m) { return c.pages + ((int64_t)page_at[m] * H + h) * size; };
  if constexpr (kMma) {
    // first the tokens' products, to the new page, then the pages are added to what its L2 lines hold: fragments of
    // the pages, 32 bytes per row, would take HBM three times as long
    tc::cp_async_wait_all();
    __syncthreads();
    const int g = lane >> 2, i = 2 * (lane & 3);
    const int mrow = (lane & 7) + ((lane >> 4) << 3), mcol = ((lane >> 3) & 1) << 3;
    for (int nt = w; nt < dv / 8; nt += kAcceptWarps) {
      uint32_t b[kW / 16][3][2];
      load_decayed(b, vs + 8 * nt, tok, vp);
      // two row tiles at a time
      for (int d = 0; d < dk; d += 32) {
        float f[2][4] = {};
#pragma unroll
        for (int v = 2; v >= 0; --v)
#pragma unroll
          for (int q = 0; q < kW / 16; ++q)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              uint32_t ka[4];  // (past the last row: of others, not stored)
              ldmatrix_trans(ka, ks + (16 * q + mrow) * kp + min(d + 16 * z, dk - 16) + mcol);
              mma_bf16(f[z], ka, b[q][v][0], b[q][v][1]);
            }
        const int64_t at = (int64_t)(d + g) * dv + 8 * nt + i;  // rows g, g + 8, g + 16, g + 24
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (d + 8 * u < dk)
            *reinterpret_cast<float2*>(D + at + 8 * u * dv) = make_float2(f[u >> 1][2 * (u & 1)], f[u >> 1][2 * (u & 1) + 1]);
      }
    }
    if (to) __syncthreads();
    for (int i0 = tid; to && i0 < size / 4; i0 += 4 * kAcceptThreads) {
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + u * kAcceptThreads < size / 4) v[u] = __ldcg(reinterpret_cast<const float4*>(D) + i0 + u * kAcceptThreads);
      for (int m = 0; m < to; m += kTogether) {
        float4 y[kTogether][4];
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (m + q < to && i0 + u * kAcceptThreads < size / 4)
              y[q][u] = __ldcs(reinterpret_cast<const float4*>(page(m + q)) + i0 + u * kAcceptThreads);
#pragma unroll
        for (int q = 0; q < kTogether; ++q)
          if (m + q < to)
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = fma4(page_e[m + q], y[q][u], v[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + u * kAcceptThreads < size / 4) reinterpret_cast<float4*>(D)[i0 + u * kAcceptThreads] = v[u];
    }
  } else {  // four rows of four columns per thread and pass
    const int groups = dv / 4, lanes = kAcceptThreads / groups, col = 4 * (tid % groups);
    for (int d = 4 * (tid / groups); tid / groups < lanes && d < dk; d += 4 * lanes) {
      float4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int m = 0; m < to; ++m)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (d + u < dk) x[u] = fma4(page_e[m], *reinterpret_cast<const float4*>(page(m) + (int64_t)(d + u) * dv + col), x[u]);
      for (int i = 0; i < kW; ++i) {
        const float4 v4 = *reinterpret_cast<const float4*>(vf + i * vp + col);
        const float4 k4 = *reinterpret_cast<const float4*>(kf + i * kp + d);
        const float e = tok[i];
        x[0] = fma4(e * k4.x, v4, x[0]);
        x[1] = fma4(e * k4.y, v4, x[1]);
        x[2] = fma4(e * k4.z, v4, x[2]);
        x[3] = fma4(e * k4.w, v4, x[3]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (d + u < dk) *reinterpret_cast<float4*>(D + (int64_t)(d + u) * dv + col) = x[u];
    }
  }
  // the path's tokens to their places: those of this block, which no fold reads there, this head's values of the
  // next one, and its keys where no other head reads them, else by the row's last CTA to have read this one's
  put_values<T>(c, a, row, s, r, path, 0, ends, h, h + 1);
  if (h % G == 0) put_keys<T>(c, a, row, s, r, path, 0, ends, hq, hq + 1);
  if (h == 0 && tid == 0) a.new_pos[row] = pos + count;
  if (count == ends) return;
  put_values<T>(c, a, row, s, r, path, ends, count, h, h + 1);
  if (G == 1) {
    put_keys<T>(c, a, row, s, r, path, ends, count, h, h + 1);
    return;
  }
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    last_s = atomicAdd(sc.done + s, 1) == H - 1;
  }
  __syncthreads();
  if (last_s) put_keys<T>(c, a, row, s, r, path, ends, count, 0, Hqk);
}

template <typename T, bool kMma>
cudaError_t launch_both(const ll_cache& c, const AcceptArgs& a, cudaStream_t s) {
  const size_t row = kMma ? sizeof(T) * (size_t)(c.dk + c.dv + 2 * kPad) : sizeof(float) * (size_t)(((c.dk + 3) & ~3) + c.dv);
  const auto kernel = accept_kernel<T, kMma>;
  cudaError_t e = allow_shared(kernel);
  if (e != cudaSuccess) return e;  // before the plan changes the tables
  accept_plan_kernel<<<1, kPlanThreads, 0, s>>>(c, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_following(true, kernel, dim3((unsigned)(a.n * c.H)), kAcceptThreads, kW * row, 1, s, c, a);
}

template <typename T>
cudaError_t launch(const ll_cache& c, const AcceptArgs& a, cudaStream_t s) {
  if constexpr (sizeof(T) == 2) {
    const int64_t all = c.dk | c.dv | a.sk[0] | a.sk[1] | a.sk[2] | a.sv[0] | a.sv[1] | a.sv[2];
    const bool whole = all % 8 == 0 && ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 15u) == 0;
    if (whole && c.dk % 16 == 0) return launch_both<T, true>(c, a, s);
  }
  return launch_both<T, false>(c, a, s);
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
