// The paged decode cache: the decode step over sequences at positions of their own, and the
// operators on its pages.
//
// After n positions a slot holds the raw tokens of its current block of 64 (n mod 64 of them)
// and, for every set bit i of j = n / 64, one page: the state of the aligned run of 2^i blocks
// that the Fenwick partition of block j has there, as it was at its last token.  What has
// decayed since is one number per page and head (page_log), brought up to date once per block;
// inside a block the tokens' own log a are summed on the fly.  So a step reads its pages but
// never rewrites them: it reads popcount(j) pages and the block's tokens, writes one token, and
// at a block's last token folds the pages below ctz(j + 1) and the block into one new page.
// The dense step reads and rewrites every level that holds data.
//
// Everything a step reads is only written by other steps: the token goes to a place that this
// step does not read, the folded page to a page that is not live, and page_log of block j to
// the copy of block j + 1's parity.  So the CTAs of one sequence need no order among them, and a
// step repeated at the same position gives the same result.
//
// A page is free when its reference count is 0, and the lowest free ones are taken first, in
// the order of the rows that ask: the result of every call is determined by its inputs.
#include <algorithm>

#include "cache_common.cuh"

namespace ll {
namespace {

// ---------------------------------------------------------------- reserve, free

// reserve (pos given): each slot keeps the pages that are live at its position and, at a
// block's last position, has the page its fold goes to.  That page is the slot's alone: one that is
// left over from earlier positions and shared is given up like the others.  free (pos null): no
// page is kept.  One CTA: the order of the rows decides who gets which page, and the work is a
// chain of a few latencies: 2 us before a step of one row, 6 before one of 128.
__global__ void __launch_bounds__(kPlanThreads) cache_reserve_kernel(ll_cache c, const int* slots,
                                                                     const int* pos, int64_t n) {
  __shared__ int slot_s[kPlanThreads];
  const Scratch sc = scratch_of(c);
  const int tid = threadIdx.x;
  let_next_start();
  if (n <= kPlanThreads) {  // a row per thread
    const int s = tid < n ? slots[tid] : -1, t = tid < n && pos ? pos[tid] : 0;
    slot_s[tid] = s;
    bool bad = s < -1 || s >= c.slots, shared = false;
    const bool ok = position_ok(c, t), fold = ok && (t & (kW - 1)) == kW - 1;
    const int e = s >= 0 && !bad && fold ? fold_page(c, s, t >> kLogW, &shared) : -1;
    __syncthreads();
    if (s >= 0)
      for (int i = 0; i < tid; ++i) bad |= slot_s[i] == s;
    if (bad) raise(c, LL_CACHE_ERR_SLOT);
    const bool named = s >= 0 && !bad;
    if (named && !ok) raise(c, LL_CACHE_ERR_POSITION);
    settle_few(c, (int)n, named && ok ? s : -1, t >> kLogW, fold, e, shared);
    return;
  }
  claim_slots(c, slots, n, sc.owner);
  for (int64_t r = tid; pos && r < n; r += kPlanThreads)
    if (owns(c, sc.owner, slots[r], r) && !position_ok(c, pos[r])) raise(c, LL_CACHE_ERR_POSITION);
  auto pos_of = [&](int64_t r) { return pos ? pos[r] : 0; };
  __syncthreads();
  settle_pages(c, n, [&](int64_t r) { return owns(c, sc.owner, slots[r], r) && position_ok(c, pos_of(r)) ? slots[r] : -1; },
               [&](int64_t r) { return pos_of(r) >> kLogW; },
               [&](int64_t r) { return (pos_of(r) & (kW - 1)) == kW - 1; });
}

// ---------------------------------------------------------------- load

// The pages of n slots that hold T positions each; the copies follow in cache_load_kernel.
__global__ void __launch_bounds__(kPlanThreads) cache_load_plan_kernel(ll_cache c,
                                                                       const int* slots,
                                                                       int64_t n, int64_t T) {
  const Scratch sc = scratch_of(c);
  const int M = (int)c.levels, j = (int)(T >> kLogW), per = __popc(j);
  let_next_start();
  claim_slots(c, slots, n, sc.owner);
  for (int64_t k = threadIdx.x; k < n * M; k += kPlanThreads) {
    const int64_t r = k / M;
    const int m = (int)(k - r * M), s = slots[r];
    if (!owns(c, sc.owner, s, r)) continue;
    int* e = c.page_table + (int64_t)s * M + m;
    if (*e >= 0) drop_page(c, *e);
    *e = -1;
  }
  if (per == 0) return;
  __syncthreads();
  int64_t rows = 0;
  for (int64_t base = 0; base < n; base += kPlanThreads) {
    const int64_t r = base + threadIdx.x;
    const bool on = r < n && owns(c, sc.owner, slots[r], r);
    int total;
    int64_t rank = (rows + block_scan(on, &total)) * per;
    if (on)
      for (int m = 0; m < M; ++m)
        if ((j >> m) & 1) {
          if (rank < c.n_pages) sc.from[rank] = (int)((int64_t)slots[r] * M + m);
          ++rank;
        }
    rows += total;
  }
  const int64_t count = rows * per;
  if (count == 0) return;
  __syncthreads();
  if (count > c.n_pages && threadIdx.x == 0) raise(c, LL_CACHE_ERR_PAGES);
  take_pages(c, sc.from, (int)min(count, c.n_pages));
}

constexpr int kCopyThreads = 256;
constexpr int kFlight = 8;  // 16-byte loads a thread has on their way: 32 KB per CTA

// dst[i] = f(src[i]) for n float4, by the CTA; src is read once, with kFlight loads in flight.
template <typename F>
__device__ __forceinline__ void copy4(float4* dst, const float4* src, int64_t n, F f) {
  for (int64_t i0 = 0; i0 < n; i0 += kFlight * kCopyThreads) {
    float4 x[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int64_t i = i0 + u * kCopyThreads + threadIdx.x;
      if (i < n) x[u] = __ldcs(src + i);
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int64_t i = i0 + u * kCopyThreads + threadIdx.x;
      if (i < n) __stcs(dst + i, f(x[u]));
    }
  }
}

// rows x width elements to dst (dense, 16-byte aligned) from src (row stride `stride`), by the CTA.
template <typename T>
__device__ __forceinline__ void copy_rows(T* dst, const T* src, int64_t stride, int rows, int width) {
  constexpr int per = 16 / sizeof(T);
  if (width % per == 0 && stride % per == 0 && (reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
    const int chunks = width / per, n = rows * chunks;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kCopyThreads) {
      const int r = i / chunks, c = i - r * chunks;
      reinterpret_cast<uint4*>(dst)[i] = *reinterpret_cast<const uint4*>(src + r * stride + c * per);
    }
  } else {
#pragma unroll 4
    for (int i = threadIdx.x; i < rows * width; i += kCopyThreads) {
      const int r = i / width;
      dst[i] = src[r * stride + (i - r * width)];
    }
  }
}

struct TokenStrides {
  int64_t k[3], v[3], a[3];  // batch, position, head
};

// blockIdx.y < per: one page of one (row, head) from the dense levels; the last: its tokens.
// T a multiple of 64: the block that ended with the prompt is folded, as the step at its last
// token would have: the levels that position T merges become the lowest page.  Bound by HBM: 32
// prompts of 12345 tokens, 16 heads, d 128: 30 us for 164 MB, 5.4 TB/s (one 16-byte copy in
// flight per thread instead of kFlight: 53 us).
template <typename T_>
__global__ void __launch_bounds__(kCopyThreads) cache_load_kernel(
    ll_cache c, const int* __restrict__ slots, int T, const float* __restrict__ state, int L,
    const T_* __restrict__ k, const T_* __restrict__ v, const float* __restrict__ log_a, int Tk,
    TokenStrides st) {
  const int H = (int)c.H, G = (int)(c.H / c.Hqk), dk = (int)c.dk, dv = (int)c.dv;
  const int64_t row = blockIdx.x / H;
  wait_for_previous();
  const int h = (int)(blockIdx.x - row * H), s = slots[row];
  if (!owns(c, scratch_of(c).owner, s, row)) return;
  const int j = T >> kLogW, r = T & (kW - 1), par = j & 1;
  const int M = (int)c.levels;
  if (blockIdx.y < gridDim.y - 1) {
    int m = 0;
    for (int left = blockIdx.y, x = j; m < M; ++m, x >>= 1)
      if ((x & 1) && left-- == 0) break;
    const int e = c.page_table[(int64_t)s * M + m];
    if (e < 0 || e >= c.n_pages) return;
    const int64_t size = (int64_t)dk * dv;
    const bool sum = r == 0 && (j & ((1 << m) - 1)) == 0;
    const int lo = sum ? 0 : kLogW + 1 + m, hi = sum ? kLogW + m : lo;
    const float4* src = reinterpret_cast<const float4*>(state + (row * H + h) * (int64_t)L * size);
    float4* dst = reinterpret_cast<float4*>(c.pages + ((int64_t)e * H + h) * size);
    const int64_t n4 = size / 4;
    if (!sum) {
      copy4(dst, src + lo * n4, n4, [](float4 x) { return x; });
    } else {
      for (int64_t i = threadIdx.x; i < n4; i += kCopyThreads) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int l = lo; l <= hi; ++l) {
          const float4 y = __ldcs(src + l * n4 + i);
          x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        __stcs(dst + i, x);
      }
    }
    if (threadIdx.x == 0) c.page_log[(((int64_t)s * 2 + par) * M + m) * H + h] = 0.f;
    return;
  }
  if (h == 0 && threadIdx.x == 0) c.page_from[s * 2 + par] = r;
  const int t0 = Tk - r;  // the block's tokens are the last r given
  copy_rows(static_cast<T_*>(c.win_v) + ((int64_t)s * H + h) * kW * dv,
            v + row * st.v[0] + t0 * st.v[1] + h * st.v[2], st.v[1], r, dv);
  if (h % G == 0)
    copy_rows(static_cast<T_*>(c.win_k) + ((int64_t)s * c.Hqk + h / G) * kW * dk,
              k + row * st.k[0] + t0 * st.k[1] + (h / G) * st.k[2], st.k[1], r, dk);
  for (int i = threadIdx.x; i < r; i += kCopyThreads)
    c.win_log_a[((int64_t)s * H + h) * kW + i] =
        log_a ? log_a[row * st.a[0] + (t0 + i) * st.a[1] + h * st.a[2]] : 0.f;
}

// ---------------------------------------------------------------- step

// An item is one (row, head).  A producer warp brings its block's tokens and then its pages, in
// stages of up to 16 KB, to shared memory by bulk copies, and eight warps consume them.  Bound by
// HBM: a page of 128 x 128 is 64 KB for 32 KFLOP.  The two forms of the kernel:
//
// queue: two persistent CTAs per SM (one alone is bound by its warps' latency: 195 us where two take
// 153 at 128 rows of position 16300).  A scheduler thread takes the grid's pending items (cluster
// launch control) and kLoaders warps bring the next items' small inputs, so that copies are in
// flight across items, and an item's loads, scores and reduction hide behind another's pages.
// 128 rows of 16 heads at positions up to 16383: 95 us for 556 MB, 5.9 TB/s; 32 rows of 48 heads
// with one q/k up to 131071: 55 us, 5.4 TB/s.  The rest is the tail: the rows of a batch
// differ by their pages and by their folds.
//
// split: for batches of fewer items than SMs.  A cluster of `split` CTAs per item, each with a
// share of the states' rows and of the block's tokens, whose first adds up their parts of the
// output (distributed shared memory); all warps load the item's inputs.  Shares of rows are
// contiguous in a page; shares of columns took twice the time for a single sequence, each of
// their rows being a copy of its own.  One sequence of 16 heads at position 12345: 5.4 us, the
// latency of a launch and of reads that wait for one another (position, table, pages, sums).
//
// bf16 tokens spill 7 words (split) and 5 words (queue) at the 80 registers that two CTAs leave.
//
// A stage is kRowsPer rows per thread of one page; the pages of a row chunk come one after the
// other, so that a fold can sum them and the tokens' products for its rows in registers.
constexpr int kConsumers = 256;
constexpr int kStepWarps = kConsumers / 32;
constexpr int kProducer = kStepWarps, kScheduler = kStepWarps + 1, kFirstLoader = kStepWarps + 2;
constexpr int kLoaders = 2;  // and items on their way
constexpr int kQueueThreads = kConsumers + 64 + 32 * kLoaders;
constexpr int kSplitThreads = kConsumers + 96;  // one loader
constexpr int kRowsPer = 4;
constexpr int kStageFloats = kConsumers * 4 * kRowsPer;
constexpr int kMaxSplit = 8;  // CTAs of a cluster
constexpr int kMaxStages = 8;

struct StepArgs {
  const int* slots;
  const int* pos;
  const void* q;
  const void* k;
  const void* v;
  const float* log_a;  // may be null
  const float* lam;
  void* out;
  int n, L, split, stages;
};

// What the warps of a CTA hand each other.
struct __align__(16) Item {
  __align__(16) float q[128];   // v and tok are read as vectors
  __align__(16) float k[128];
  __align__(16) float v[128];
  __align__(16) float tok[kW];  // decay from each token of the block to the new one
  float lam[kMaxLevels + kLogW + 1];
  // the live pages, lowest level first: log decay, decay, decay times lambda
  float page_log[kMaxLevels], page_e[kMaxLevels], page_w[kMaxLevels];
  int page_at[kMaxLevels], page_lv[kMaxLevels];
  int kind, row, h, slot, pos, dest;  // kind: kRun, kSkip or kStop
  unsigned why;                       // (split) what load_links found
  float log_a;
};
enum { kRun, kSkip, kStop };

struct StepSmem {
  Item item[kLoaders];
  __align__(16) float parts[kMaxSplit][128];
  float4 red[kConsumers];
  float p[kW], self;
  int index[kLoaders];          // the items the loaders are to bring
  __align__(16) uint4 next;     // cluster launch control's answer
  uint64_t index_full[kLoaders], index_empty[kLoaders], item_full[kLoaders], item_empty[kLoaders];
  uint64_t window_full, window_empty, answered;
  uint64_t full[kMaxStages], empty[kMaxStages];
};

// Asks for a pending CTA of the grid in this one's stead; the answer goes to *to.
__device__ __forceinline__ void ask_next(uint4* to, uint64_t* bar) {
  tc::mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          tc::smem_u32(to)),
      "r"(tc::smem_u32(bar))
      : "memory");
}
// The CTA's index, or -1 where none was pending.
__device__ __forceinline__ int read_next(const uint4* from) {
  uint32_t got, x = 0;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, r;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(tc::smem_u32(from))
      : "memory");
  tc::fence_proxy_async_smem();  // the next answer is written behind this read
  return got ? (int)x : -1;
}

// The item's vectors, by thread i0 of kStep: all loads first (fetch), for a loader warp's time is
// the latency of its loads, one after the other or all at once; then to shared memory (put).
template <typename T, int kStep>
struct Vectors {
  static constexpr int N = kStep < 128 ? 128 / kStep : 1;
  T q[N], k[N], v[N];
  float lam;
  bool twice;  // an earlier row has its slot
  __device__ __forceinline__ void fetch(const ll_cache& c, const StepArgs& a, int row, int h, int s, int i0) {
    const int Hqk = (int)c.Hqk, G = (int)c.H / Hqk, dk = (int)c.dk, dv = (int)c.dv;
    const int64_t bh = (int64_t)row * (int)c.H + h;
    const T* gq = static_cast<const T*>(a.q) + ((int64_t)row * Hqk + h / G) * dk;
    const T* gk = static_cast<const T*>(a.k) + ((int64_t)row * Hqk + h / G) * dk;
    const T* gv = static_cast<const T*>(a.v) + bh * dv;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int i = i0 + u * kStep;
      if (i < dk) {
        q[u] = gq[i];
        k[u] = gk[i];
      }
      if (i < dv) v[u] = gv[i];
    }
    if (i0 < (int)c.levels + kLogW + 1) lam = a.lam[bh * a.L + i0];
    twice = false;
#pragma unroll 4
    for (int i = i0; i < row; i += kStep) twice |= a.slots[i] == s;
  }
  __device__ __forceinline__ void put(const ll_cache& c, int i0, Item& it) const {
    const int dk = (int)c.dk, dv = (int)c.dv;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int i = i0 + u * kStep;
      if (i < dk) {
        it.q[i] = to_f32(q[u]);
        it.k[i] = to_f32(k[u]);
      }
      if (i < dv) it.v[i] = to_f32(v[u]);
    }
    if (i0 < (int)c.levels + kLogW + 1) it.lam[i0] = lam;
  }
};

// The item's decays and pages, by one warp; s and t are fine.  Returns why the row cannot be served.
__device__ __forceinline__ unsigned load_links(const ll_cache& c, const StepArgs& a, int row, int h, int s,
                                           int t, Item& it) {
  const int lane = threadIdx.x & 31, H = (int)c.H, M = (int)c.levels;
  const int64_t bh = (int64_t)row * H + h;
  const int j = t >> kLogW, r = t & (kW - 1), par = j & 1;
  const int to = r == kW - 1 ? __ffs(j + 1) - 1 : -1;
  const bool here = lane < M && (j >> lane) & 1;
  const int e = here || lane == to ? c.page_table[(int64_t)s * M + lane] : 0;
  // a fold writes only to a page of the slot's own
  const bool shared = lane == to && e >= 0 && e < c.n_pages && c.refcount[e] != 1;
  const float log = here ? c.page_log[(((int64_t)s * 2 + par) * M + lane) * H + h] : 0.f;
  const float la = a.log_a ? a.log_a[bh] : 0.f;
  const float lam = here ? a.lam[bh * a.L + kLogW + 1 + lane] : 0.f;
  const float* wa = c.win_log_a + ((int64_t)s * H + h) * kW;
  const float x0 = lane < r ? wa[lane] : 0.f, x1 = lane + 32 < r ? wa[lane + 32] : 0.f;
  const int from = c.page_from[s * 2 + par];
  float since;
  block_decays(x0, x1, r, from, it.tok, &since);
  it.tok[lane] = expf(it.tok[lane] + la);
  it.tok[lane + 32] = lane + 32 == r ? 1.f : expf(it.tok[lane + 32] + la);  // a fold's own token: 1
  if (here) {
    const int at = __popc(j & ((1 << lane) - 1));
    it.page_at[at] = e;
    it.page_lv[at] = lane;
    it.page_log[at] = log + since + la;
    it.page_e[at] = expf(log + since + la);
    it.page_w[at] = it.page_e[at] * lam;
  }
  if (lane == to) it.dest = e;
  if (lane == 0) {
    it.log_a = la;
    it.row = row;
    it.h = h;
    it.slot = s;
    it.pos = t;
  }
  if (__any_sync(0xffffffffu, e < 0 || e >= c.n_pages || shared)) return LL_CACHE_ERR_MISSING;
  return j && from > r ? LL_CACHE_ERR_POSITION : 0;  // (as before_pages)
}

constexpr int kPad = 8;  // elements

// An item's geometry in a CTA: its state rows [k0, k1) and tokens [t0, t1).  A fold needs all
// tokens' products, so it brings them all ([b0, b1)).
struct Part {
  int j, r, to, live;
  bool fold, mma;  // mma: the fold's token products come from the tensor cores
  int k0, k1, t0, t1, b0, b1;
  int kp, vp;      // elements from token to token in the window: set off by 16 bytes for mma
};
template <typename T>
__device__ __forceinline__ Part part_of(int pos, int dk, int dv, int Z, int sp) {
  Part p;
  p.j = pos >> kLogW;
  p.r = pos & (kW - 1);
  p.fold = p.r == kW - 1;
  p.to = p.fold ? __ffs(p.j + 1) - 1 : -1;  // the level the block is folded to
  p.live = __popc(p.j);
  const int share = (dk + Z - 1) / Z;
  p.k0 = min(dk, sp * share);
  p.k1 = min(dk, p.k0 + share);
  const int tokens = ((p.r + Z - 1) / Z + 7) & ~7;  // whole 16-byte pieces, whatever the row
  p.t0 = min(p.r, sp * tokens);
  p.t1 = min(p.r, p.t0 + tokens);
  p.b0 = p.fold ? 0 : p.t0;
  p.b1 = p.fold ? p.r : p.t1;
  // tensor cores: bf16 tokens whose rows are whole 16-byte pieces
  p.mma = sizeof(T) == 2 && p.fold && dk % 8 == 0 && dv % 8 == 0 && p.k0 % 8 == 0 &&
          (p.k1 - p.k0) % 16 == 0;
  p.kp = p.mma ? dk + kPad : dk;
  p.vp = p.mma ? dv + kPad : dv;
  return p;
}

__device__ __forceinline__ void consumer_sync() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(kConsumers) : "memory");
}
// Whether x is true in any consumer.
__device__ __forceinline__ bool consumer_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(kConsumers)
      : "memory");
  return r != 0;
}

// The products of a fold's 64 tokens for state rows [k0, k1) (a multiple of 16), by the consumer
// warps, to D [dk][dv]: sum over s of k_s (e_s v_s)^T on the tensor cores, bf16 keys as they are
// and e v split into three bf16 parts, which together are its fp32 value; products and sums
// are fp32.  (Multiply-adds took 10 us more per fold, the tail of a ragged batch.)  Infinities come
// out as in the sum itself, where the parts' products are all of one sign: the parts are cut off
// towards zero, and what is left of a value that is not 0 is never 0 or NaN (infinity less
// itself) but at least the least bf16, whose product with a key is below any normal number.
__device__ __forceinline__ void fold_tokens(const __nv_bfloat16* wks, const __nv_bfloat16* wvs,
                                            const float* tok, int kp, int vp, int dv, int k0, int k1,
                                            float* D) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int g = lane >> 2, i = 2 * (lane & 3);
  // ldmatrix rows: lanes 0-7, 8-15, 16-23, 24-31 address the four 8 x 8 matrices
  const int mrow = (lane & 7) + ((lane >> 4) << 3), mcol = ((lane >> 3) & 1) << 3;
  for (int nt = w; nt < dv / 8; nt += kStepWarps) {
    uint32_t b[kW / 16][3][2];
    load_decayed(b, wvs + 8 * nt, tok, vp);
    for (int d = k0; d < k1; d += 16) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < kW / 16; ++ks) {
        uint32_t a[4];
        ldmatrix_trans(a, wks + (16 * ks + mrow) * kp + d + mcol);
#pragma unroll
        for (int v = 2; v >= 0; --v) mma_bf16(c, a, b[ks][v][0], b[ks][v][1]);
      }
      *reinterpret_cast<float2*>(D + (d + g) * dv + 8 * nt + i) = make_float2(c[0], c[1]);
      *reinterpret_cast<float2*>(D + (d + g + 8) * dv + 8 * nt + i) = make_float2(c[2], c[3]);
    }
  }
}

template <typename T, typename OutT, bool kQueue>
__global__ void __launch_bounds__(kQueue ? kQueueThreads : kSplitThreads, 2)
    cache_step_kernel(ll_cache c, StepArgs a) {
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ StepSmem sm;
  const int H = (int)c.H, Hqk = (int)c.Hqk, G = H / Hqk, dk = (int)c.dk, dv = (int)c.dv, M = (int)c.levels;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int Z = kQueue ? 1 : a.split, sp = kQueue ? 0 : blockIdx.x % Z;  // the CTA's rank in its cluster
  const int groups = dv >> 2, lanes = kConsumers / groups;  // column groups, threads down the rows
  const int per = min(kRowsPer, ((dk + Z - 1) / Z + lanes - 1) / lanes);  // rows of a thread in a stage
  const int span = per * lanes;
  float* ring = reinterpret_cast<float*>(dyn);
  T* wks = reinterpret_cast<T*>(dyn + (size_t)a.stages * kStageFloats * 4);
  T* wvs = wks + kW * (dk + kPad);
  if (tid == 0) {
    for (int i = 0; i < kLoaders; ++i) {
      tc::mbar_init(&sm.index_full[i], 1);
      tc::mbar_init(&sm.index_empty[i], 1);
      tc::mbar_init(&sm.item_full[i], 1);
      tc::mbar_init(&sm.item_empty[i], kStepWarps + 1);  // the consumers and the producer
    }
    tc::mbar_init(&sm.window_full, 1);
    tc::mbar_init(&sm.window_empty, kStepWarps);
    tc::mbar_init(&sm.answered, 1);
    for (int i = 0; i < a.stages; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.empty[i], kStepWarps);
    }
    tc::fence_mbar_init();
  }
  wait_for_previous();
  // the block's tokens [b0, b1): whole rows from a multiple of 8 rows on, so 16-byte aligned; the
  // length is rounded up to 16 bytes, still inside the window.  Without tokens the barrier takes
  // an empty phase.
  auto bring_window = [&](int64_t s, int h, const Part& g) {
    const uint32_t nk = ((g.b1 - g.b0) * dk * sizeof(T) + 15) & ~15u;
    const uint32_t nv = ((g.b1 - g.b0) * dv * sizeof(T) + 15) & ~15u;
    const T* wk = static_cast<const T*>(c.win_k) + (s * Hqk + h / G) * kW * dk;
    const T* wv = static_cast<const T*>(c.win_v) + (s * H + h) * kW * dv;
    tc::mbar_arrive_expect_tx(&sm.window_full, nk + nv);  // (mma: rows of whole 16 bytes, no rounding)
    if (g.mma) {
      for (int i = g.b0; i < g.b1; ++i) {
        bulk_load(wks + i * g.kp, wk + i * dk, dk * sizeof(T), &sm.window_full);
        bulk_load(wvs + i * g.vp, wv + i * dv, dv * sizeof(T), &sm.window_full);
      }
    } else if (g.b1 > g.b0) {
      bulk_load(wks + g.b0 * dk, wk + g.b0 * dk, nk, &sm.window_full);
      bulk_load(wvs + g.b0 * dv, wv + g.b0 * dv, nv, &sm.window_full);
    }
  };
  bool ok = true, brought = false;
  if (kQueue) {
    __syncthreads();
  } else {
    if (Z > 1) cluster_arrive();  // this CTA is there
    const int index = blockIdx.x / Z, row = index / H, h = index - row * H, s = a.slots[row], t = a.pos[row];
    const unsigned bad = s == -1 ? 0 : row_bad(c, s, t);
    const bool run = s != -1 && !bad;
    __syncthreads();  // the barriers are there
    bool twice = false;
    if (run) {
      if (w == kProducer) {
        if (lane == 0) bring_window(s, h, part_of<T>(t, dk, dv, Z, sp));
        brought = true;
      } else if (w == kScheduler + 1) {
        const unsigned why = load_links(c, a, row, h, s, t, sm.item[0]);
        if (lane == 0) sm.item[0].why = why;
      } else if (w < kStepWarps) {
        Vectors<T, kConsumers> x;
        x.fetch(c, a, row, h, s, tid);
        x.put(c, tid, sm.item[0]);
        twice = x.twice;
      }
    }
    twice = __syncthreads_or(twice);
    if (tid == 0) {
      const unsigned why = bad ? bad : twice ? LL_CACHE_ERR_SLOT : run ? sm.item[0].why : 0;
      if (why && sp == 0 && h == 0) raise(c, why);
      sm.item[0].kind = run && !why ? kRun : kSkip;
    }
    __syncthreads();
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (kQueue && w >= kFirstLoader) {
    const int L = w - kFirstLoader;
    Item& it = sm.item[L];
    for (int turn = 0;; turn ^= 1) {
      ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&sm.index_full[L], turn));
      if (!ok) break;
      const int index = sm.index[L];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.index_empty[L]);
      ok = __all_sync(0xffffffffu, tc::mbar_wait_short(&sm.item_empty[L], turn ^ 1));
      if (!ok) break;
      int kind = kStop;
      if (index >= 0) {
        const int row = index / H, h = index - row * H, s = a.slots[row], t = a.pos[row];
        kind = kSkip;
        if (s != -1) {
          unsigned why = row_bad(c, s, t);
          if (!why) {
            Vectors<T, 32> x;
            x.fetch(c, a, row, h, s, lane);
            why = load_links(c, a, row, h, s, t, it);
            x.put(c, lane, it);
            if (__any_sync(0xffffffffu, x.twice)) why = LL_CACHE_ERR_SLOT;
          }
          if (!why) kind = kRun;
          else if (lane == 0 && h == 0) raise(c, why);
        }
      }
      if (lane == 0) it.kind = kind;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.item_full[L]);
      if (index < 0) break;
    }
    if (!ok && lane == 0) raise(c, LL_CACHE_ERR_WAIT);
  } else if (kQueue && w == kScheduler) {
    if (lane == 0) {
      int next = blockIdx.x, after = -1;  // after: loaders that have been told to stop
      for (int n = 0, L = 0, turn = 0; ok && after < kLoaders - 1; ++n) {
        if (next >= 0) ask_next(&sm.next, &sm.answered);
        ok = tc::mbar_wait_short(&sm.index_empty[L], turn ^ 1);
        sm.index[L] = next;
        tc::mbar_arrive(&sm.index_full[L]);
        if (next < 0) {
          ++after;
        } else {
          const bool got = tc::mbar_wait_short(&sm.answered, n & 1);
          ok = ok && got;
          next = got ? read_next(&sm.next) : -1;
        }
        if (++L == kLoaders) {
          L = 0;
          turn ^= 1;
        }
      }
      if (!ok) raise(c, LL_CACHE_ERR_WAIT);
    }
    __syncwarp();
  } else if (w == kProducer) {
    int st = 0, phase = 0, ib = 0, turn = 0, used = brought ? 1 : 0;
    while (lane == 0) {
      if (kQueue && !(ok = tc::mbar_wait_short(&sm.item_full[ib], turn))) break;
      const Item& it = sm.item[ib];
      if (it.kind == kStop || (!kQueue && it.kind == kSkip)) break;
      if (it.kind == kRun) {
        const Part g = part_of<T>(it.pos, dk, dv, Z, sp);
        const int h = it.h;
        if (kQueue) {
          if (!(ok = tc::mbar_wait_short(&sm.window_empty, (used & 1) ^ 1))) break;
          bring_window(it.slot, h, g);
          ++used;
        }
        for (int d0 = g.k0; d0 < g.k1 && ok; d0 += span) {
          const int bytes = min(span, g.k1 - d0) * dv * 4;
          for (int m = 0; m < g.live; ++m) {
            if (!(ok = tc::mbar_wait_short(&sm.empty[st], phase ^ 1))) break;
            tc::mbar_arrive_expect_tx(&sm.full[st], bytes);
            bulk_load(ring + st * kStageFloats,
                      c.pages + (((int64_t)it.page_at[m] * H + h) * dk + d0) * dv, bytes, &sm.full[st]);
            if (++st == a.stages) {
              st = 0;
              phase ^= 1;
            }
          }
        }
        if (!ok) break;
      }
      if (!kQueue) break;
      tc::mbar_arrive(&sm.item_empty[ib]);
      if (++ib == kLoaders) {
        ib = 0;
        turn ^= 1;
      }
    }
    if (lane == 0 && !ok) raise(c, LL_CACHE_ERR_WAIT);
    if (lane == 0 && (!ok || !kQueue)) {  // the copies on their way end before the CTA does
      for (int i = 0; i < a.stages; ++i)  // each stage's last use (none: the barrier is fresh)
        tc::mbar_wait_short(&sm.full[i], i < st ? phase : phase ^ 1);
      tc::mbar_wait_short(&sm.window_full, (used & 1) ^ 1);
    }
    __syncwarp();
  } else if (w < kStepWarps) {
    const int cg = tid % groups, row0 = tid / groups;
    const bool on = row0 < lanes;
    int st = 0, phase = 0;
    int ib = 0, turn = 0, used = 0;  // item buffer, its phase; items with a window so far
    for (;;) {
      if (kQueue) {
        // one wait that ran out of time ends the CTA's work, in all warps alike
        ok = tc::mbar_wait_short(&sm.item_full[ib], turn) && ok;
        if (consumer_any(!ok)) {
          ok = false;
          break;
        }
      }
      const Item& it = sm.item[ib];
      if (it.kind == kStop) break;
      if (it.kind == kSkip) {
        if (!kQueue) break;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.item_empty[ib]);
        if (++ib == kLoaders) {
          ib = 0;
          turn ^= 1;
        }
        continue;
      }
      const Part g = part_of<T>(it.pos, dk, dv, Z, sp);
      ok = tc::mbar_wait_short(&sm.window_full, used & 1) && ok;
      ++used;
      if (g.mma) {  // the new token joins the others
        if (tid < dk) wks[(kW - 1) * g.kp + tid] = from_f32<T>(it.k[tid]);
        if (tid < dv) wvs[(kW - 1) * g.vp + tid] = from_f32<T>(it.v[tid]);
      }
      // scores of the CTA's tokens, a warp every eighth; the cluster's first has the new one too
      float qv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) qv[u] = lane + 32 * u < dk ? it.q[lane + 32 * u] : 0.f;
#pragma unroll 4
      for (int i = g.t0 + w; i < g.t1; i += kStepWarps) {
        float x = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (lane + 32 * u < dk) x = fmaf(qv[u], to_f32(wks[i * g.kp + lane + 32 * u]), x);
        x = warp_sum(x);
        if (lane == 0) sm.p[i] = it.lam[fenwick_level(g.r, i)] * it.tok[i] * x;
      }
      if (w == 0 && (kQueue || sp == 0)) {
        float x = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (lane + 32 * u < dk) x = fmaf(qv[u], it.k[lane + 32 * u], x);
        x = warp_sum(x);
        if (lane == 0) sm.self = it.lam[0] * x;
      }
      consumer_sync();
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 v4 = *reinterpret_cast<const float4*>(it.v + 4 * cg);
      if (on) {
        if (row0 == 0 && (kQueue || sp == 0)) acc = fma4(sm.self, v4, acc);
#pragma unroll 4
        for (int i = g.t0 + row0; i < g.t1; i += lanes) acc = fma4(sm.p[i], load4(wvs + i * g.vp + 4 * cg), acc);
      }
      const int h = it.h;
      const int64_t bh = (int64_t)it.row * H + h;
      float* folded = c.pages + ((int64_t)it.dest * H + h) * dk * dv;  // (g.fold)
      if constexpr (sizeof(T) == 2) {
        if (g.mma) {
          fold_tokens(wks, wvs, it.tok, g.kp, g.vp, dv, g.k0, g.k1, folded);
          tc::fence_proxy_async_smem();  // the next bulk copy is written behind the new token
          consumer_sync();
        }
      }
      if (kQueue && (!g.fold || g.mma)) {  // the next item's tokens may come
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.window_empty);
      }
      for (int c0 = g.k0; c0 < g.k1; c0 += span) {
        const int d0 = c0 + per * row0;
        const int rows = on ? min(per, g.k1 - d0) : 0;  // this thread's rows (below 1: none)
        float qr[kRowsPer];
#pragma unroll
        for (int x = 0; x < kRowsPer; ++x) qr[x] = x < rows ? it.q[d0 + x] : 0.f;
        const float* mine = ring + per * row0 * dv + 4 * cg;
        if (!g.fold) {
          for (int m = 0; m < g.live; ++m) {
            ok = tc::mbar_wait_short(&sm.full[st], phase) && ok;
            const float* P = mine + st * kStageFloats;
            float4 part = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < kRowsPer; ++x)
              if (x < rows) part = fma4(qr[x], *reinterpret_cast<const float4*>(P + x * dv), part);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sm.empty[st]);
            acc = fma4(it.page_w[m], part, acc);
            if (++st == a.stages) {
              st = 0;
              phase ^= 1;
            }
          }
          continue;
        }
        float4 sum[kRowsPer];
        float4* D = reinterpret_cast<float4*>(folded + d0 * dv + 4 * cg);
#pragma unroll
        for (int x = 0; x < kRowsPer; ++x)
          sum[x] = g.mma && x < rows ? __ldcg(D + x * groups) : make_float4(0.f, 0.f, 0.f, 0.f);
        for (int m = 0; m < g.live; ++m) {
          ok = tc::mbar_wait_short(&sm.full[st], phase) && ok;
          const float* P = mine + st * kStageFloats;
          const float e = it.page_lv[m] < g.to ? it.page_e[m] : 0.f;
          float4 part = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int x = 0; x < kRowsPer; ++x)
            if (x < rows) {
              const float4 y = *reinterpret_cast<const float4*>(P + x * dv);
              part = fma4(qr[x], y, part);
              if (it.page_lv[m] < g.to) sum[x] = fma4(e, y, sum[x]);
            }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.empty[st]);
          acc = fma4(it.page_w[m], part, acc);
          if (++st == a.stages) {
            st = 0;
            phase ^= 1;
          }
        }
        if (rows > 0) {
          const bool quads = rows == 4 && dk % 4 == 0 && d0 % 4 == 0;  // four keys in one load
          for (int i = 0; i < g.r && !g.mma; ++i) {
            const float4 y = load4(wvs + i * dv + 4 * cg);
            const float e = it.tok[i];
            const T* kr = wks + i * dk + d0;
            float4 k4;
            if (quads) {
              k4 = load4(kr);
            } else {
              k4.x = to_f32(kr[0]);
              k4.y = rows > 1 ? to_f32(kr[1]) : 0.f;
              k4.z = rows > 2 ? to_f32(kr[2]) : 0.f;
              k4.w = rows > 3 ? to_f32(kr[3]) : 0.f;
            }
            sum[0] = fma4(e * k4.x, y, sum[0]);
            sum[1] = fma4(e * k4.y, y, sum[1]);
            sum[2] = fma4(e * k4.z, y, sum[2]);
            sum[3] = fma4(e * k4.w, y, sum[3]);
          }
#pragma unroll
          for (int x = 0; x < kRowsPer; ++x)
            if (x < rows && ok) D[x * groups] = g.mma ? sum[x] : fma4(it.k[d0 + x], v4, sum[x]);
        }
      }
      if (kQueue && g.fold && !g.mma) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.window_empty);
      }
      sm.red[tid] = acc;
      consumer_sync();
      if (tid < groups) {
        acc = sm.red[tid];
#pragma unroll 4
        for (int i = 1; i < lanes; ++i) acc = add4(acc, sm.red[tid + i * groups]);
        if (kQueue) store_out<OutT>(a.out, bh * dv + 4 * tid, acc);
      }
      // this token joins the block
      if (kQueue || sp == Z - 1) {
        const int64_t s = it.slot;  // q, k and v are exact in fp32: back to T they are what they were
        if (tid < dv) static_cast<T*>(c.win_v)[((s * H + h) * kW + g.r) * dv + tid] = from_f32<T>(it.v[tid]);
        if (h % G == 0 && tid < dk)
          static_cast<T*>(c.win_k)[((s * Hqk + h / G) * kW + g.r) * dk + tid] = from_f32<T>(it.k[tid]);
        if (tid == 0) c.win_log_a[(s * H + h) * kW + g.r] = it.log_a;
        if (g.fold) {  // what the next block's steps read
          const int par = (g.j & 1) ^ 1;
          if (tid < g.live && it.page_lv[tid] > g.to)
            c.page_log[((s * 2 + par) * M + it.page_lv[tid]) * H + h] = it.page_log[tid];
          if (tid == 0) {
            c.page_log[((s * 2 + par) * M + g.to) * H + h] = 0.f;
            if (h == 0) c.page_from[s * 2 + par] = 0;
          }
        }
      }
      if (!kQueue) break;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.item_empty[ib]);
      if (++ib == kLoaders) {
        ib = 0;
        turn ^= 1;
      }
    }
    if (!ok && lane == 0) raise(c, LL_CACHE_ERR_WAIT);
  }
  if (!kQueue) {
    const bool run = sm.item[0].kind == kRun;
    if (Z > 1) {
      __syncwarp();
      cluster_wait();  // all CTAs are there
      if (run && tid < groups) store_remote4(&sm.parts[sp][4 * tid], 0, acc);
      __syncwarp();
      cluster_arrive();
      cluster_wait();
      if (run && sp == 0 && tid < groups) {
        acc = *reinterpret_cast<const float4*>(&sm.parts[0][4 * tid]);
        for (int z = 1; z < Z; ++z)
          acc = add4(acc, *reinterpret_cast<const float4*>(&sm.parts[z][4 * tid]));
      }
    }
    if (run && sp == 0 && tid < groups) store_out<OutT>(a.out, ((int64_t)sm.item[0].row * H + sm.item[0].h) * dv + 4 * tid, acc);
  }
}

// ---------------------------------------------------------------- store

// One CTA per (row, head, level): the dense state's level, from a page or from the tokens, which
// are products of at most 32 (a block's levels), summed in registers from shared memory.  Bound
// by HBM: the dense levels are all written, the empty ones as zeros.  16 slots of 16 heads, L 15:
// 54 us for 343 MB, 6.4 TB/s.
template <typename T>
__global__ void __launch_bounds__(kCopyThreads) cache_store_kernel(
    ll_cache c, const int* __restrict__ slots, const int* __restrict__ pos,
    float* __restrict__ state, int L) {
  __shared__ float tok[kW], since_s;
  __shared__ __align__(16) float ks[kW / 2][128], vs[kW / 2][128];  // a level's tokens, keys decayed
  const int H = (int)c.H, G = (int)(c.H / c.Hqk), dk = (int)c.dk, dv = (int)c.dv;
  const int M = (int)c.levels, tid = threadIdx.x, level = blockIdx.y;
  const int64_t row = blockIdx.x / H;
  const int h = (int)(blockIdx.x - row * H), s = slots[row], n = pos[row];
  if (s == -1) return;
  unsigned bad = s < 0 || s >= c.slots ? LL_CACHE_ERR_SLOT : 0;
  if (!bad && (n < 0 || n > ((int64_t)kW << M) - 1)) bad = LL_CACHE_ERR_POSITION;
  const int j = n >> kLogW, r = n & (kW - 1), par = j & 1;
  // a level without its page leaves out the whole row: every warp of it looks at all of them, a
  // level per lane (a block barrier instead: 56.2 us)
  const int lane = tid & 31;
  int held = 0;
  if (!bad && lane < M && (j >> lane & 1)) {
    held = c.page_table[(int64_t)s * M + lane];
    const bool before = before_pages(c, s, n);
    if (held < 0 || held >= c.n_pages) bad = LL_CACHE_ERR_MISSING;
    else if (before) bad = LL_CACHE_ERR_POSITION;
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (bad && tid < 32 && h == 0 && level == 0) raise(c, bad);
    return;
  }
  const int64_t size = (int64_t)dk * dv, n4 = size / 4;
  float4* dst = reinterpret_cast<float4*>(state + ((row * H + h) * (int64_t)L + level) * size);
  // a page i is level 7 + i; after a whole block the lowest one holds the sum of the levels that
  // the next step merges, and stands in the highest of them
  const int low = r == 0 && j ? __ffs(j) - 1 : -1;
  const int m = low >= 0 && level == kLogW + low ? low : level - kLogW - 1;
  const bool page = m >= 0 && m < M && (j >> m & 1) && !(m == low && level != kLogW + low);
  // else tokens lo .. hi - 1 of the block, as seen from its last one
  int lo = 0, hi = 0;
  if (!page && r > 0 && level <= kLogW) {
    const int last = r - 1;
    if (level == 0) {
      lo = last;
      hi = r;
    } else if (last >> (level - 1) & 1) {
      lo = ((last >> (level - 1)) - 1) << (level - 1);
      hi = lo + (1 << (level - 1));
    }
  }
  if (!page && lo == hi) {
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t i = tid; i < n4; i += kCopyThreads) __stcs(dst + i, zero);
    return;
  }
  const int e = __shfl_sync(0xffffffffu, held, m & 31);  // (page: m < M)
  const float log = page ? c.page_log[(((int64_t)s * 2 + par) * M + m) * H + h] : 0.f;
  if (tid < 32)
    block_decays(c.win_log_a + ((int64_t)s * H + h) * kW, r, c.page_from[s * 2 + par], tok, &since_s);
  __syncthreads();
  if (page) {
    const float f = expf(log + since_s);
    const float4* src = reinterpret_cast<const float4*>(c.pages + ((int64_t)e * H + h) * size);
    copy4(dst, src, n4, [f](float4 x) { return make_float4(f * x.x, f * x.y, f * x.z, f * x.w); });
    return;
  }
  const T* wk = static_cast<const T*>(c.win_k) + (((int64_t)s * c.Hqk + h / G) * kW + lo) * dk;
  const T* wv = static_cast<const T*>(c.win_v) + (((int64_t)s * H + h) * kW + lo) * dv;
  const int n_tok = hi - lo;
#pragma unroll 4
  for (int i = tid; i < n_tok * dk; i += kCopyThreads) {
    const int u = i / dk;
    ks[u][i - u * dk] = expf(tok[lo + u]) * to_f32(wk[i]);
  }
#pragma unroll 4
  for (int i = tid; i < n_tok * dv; i += kCopyThreads) {
    const int u = i / dv;
    vs[u][i - u * dv] = to_f32(wv[i]);
  }
  __syncthreads();
  // four rows of four columns per thread and pass
  const int groups = dv / 4, lanes = kCopyThreads / groups, col = 4 * (tid % groups);
  for (int d = 4 * (tid / groups); tid / groups < lanes && d < dk; d += 4 * lanes) {
    float4 x[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) x[y] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int u = 0; u < n_tok; ++u) {
      const float4 v4 = *reinterpret_cast<const float4*>(&vs[u][col]);
      const float4 k4 = *reinterpret_cast<const float4*>(&ks[u][d]);  // (past dk: not stored)
      x[0] = fma4(k4.x, v4, x[0]);
      x[1] = fma4(k4.y, v4, x[1]);
      x[2] = fma4(k4.z, v4, x[2]);
      x[3] = fma4(k4.w, v4, x[3]);
    }
#pragma unroll
    for (int y = 0; y < 4; ++y)
      if (d + y < dk) __stcs(dst + ((int64_t)(d + y) * dv + col) / 4, x[y]);
  }
}

// ---------------------------------------------------------------- fork

// A row is left out where its target is not its own, its source is not a slot or is some row's
// target, its position is outside the cache or one that its pages are past, or a page that it needs of its source is not there.
// owner: the targets' rows, ~row of those that are left out, kNone for sources.
__device__ __forceinline__ unsigned fork_bad(const ll_cache& c, const int* owner, int s, int t) {
  if (s < 0 || s >= c.slots || __ldcg(owner + s) != kNone) return LL_CACHE_ERR_SLOT;
  return t < 0 || t > ((int64_t)kW << c.levels) - 1 ? LL_CACHE_ERR_POSITION : 0;
}

__global__ void __launch_bounds__(kPlanThreads) cache_fork_plan_kernel(ll_cache c, const int* src,
                                                                       const int* dst,
                                                                       const int* pos, int64_t n) {
  const Scratch sc = scratch_of(c);
  const int M = (int)c.levels;
  let_next_start();
  for (int64_t r = threadIdx.x; r < n; r += kPlanThreads)
    if (src[r] >= 0 && src[r] < c.slots) sc.owner[src[r]] = kNone;
  __syncthreads();
  claim_slots(c, dst, n, sc.owner, src);
  __syncthreads();
  // nothing changes before it is settled which rows are served
  for (int64_t k = threadIdx.x; k < n * M; k += kPlanThreads) {
    const int64_t r = k / M;
    const int m = (int)(k - r * M), s = src[r], d = dst[r], t = pos[r];
    if (s == -1 || d < 0 || d >= c.slots) continue;
    const int o = __ldcg(sc.owner + d);
    if (o != r && o != ~(int)r) continue;
    unsigned bad = fork_bad(c, sc.owner, s, t);
    if (bad) {
      if (m == 0) raise(c, bad);
    } else if ((t >> kLogW) >> m & 1) {
      const int page = c.page_table[(int64_t)s * M + m];
      const bool before = before_pages(c, s, t);
      if (page < 0 || page >= c.n_pages) raise(c, bad = LL_CACHE_ERR_MISSING);
      else if (before) raise(c, bad = LL_CACHE_ERR_POSITION);
    }
    if (bad) sc.owner[d] = ~(int)r;
  }
  __syncthreads();
  // every target gives up its pages and takes a share of its source's (which is no target)
  for (int64_t k = threadIdx.x; k < n * M; k += kPlanThreads) {
    const int64_t r = k / M;
    const int m = (int)(k - r * M), s = src[r], d = dst[r], t = pos[r];
    if (s == -1 || !owns(c, sc.owner, d, r)) continue;  // (-1: nobody's owner was settled here)
    int* e = c.page_table + (int64_t)d * M + m;
    const int page = (t >> kLogW) >> m & 1 ? c.page_table[(int64_t)s * M + m] : -1;
    drop_page(c, *e);
    if (page >= 0) atomicAdd(c.refcount + page, 1);
    *e = page;
  }
}

// One CTA per (row, head): the tokens of the source's block, and its pages' decays; the pages
// themselves are shared.  16 slots to 4 copies each: 13 us for 41 MB with the plan, which is a chain
// of reads that wait for one another (slots, owners, tables, counts: more than half of it).
template <typename T>
__global__ void __launch_bounds__(kCopyThreads) cache_fork_kernel(ll_cache c,
                                                                  const int* __restrict__ src,
                                                                  const int* __restrict__ dst,
                                                                  const int* __restrict__ pos) {
  const int H = (int)c.H, G = (int)(c.H / c.Hqk), dk = (int)c.dk, dv = (int)c.dv;
  const int M = (int)c.levels, tid = threadIdx.x;
  const int64_t row = blockIdx.x / H;
  wait_for_previous();
  const int h = (int)(blockIdx.x - row * H), s = src[row], d = dst[row], t = pos[row];
  const int* owner = scratch_of(c).owner;
  if (s == -1 || !owns(c, owner, d, row)) return;
  const int j = t >> kLogW, r = t & (kW - 1), par = j & 1;
  copy_rows(static_cast<T*>(c.win_v) + ((int64_t)d * H + h) * kW * dv,
            static_cast<const T*>(c.win_v) + ((int64_t)s * H + h) * kW * dv, r * dv, 1, r * dv);
  if (h % G == 0)
    copy_rows(static_cast<T*>(c.win_k) + ((int64_t)d * c.Hqk + h / G) * kW * dk,
              static_cast<const T*>(c.win_k) + ((int64_t)s * c.Hqk + h / G) * kW * dk, r * dk, 1, r * dk);
  for (int i = tid; i < r; i += kCopyThreads)
    c.win_log_a[((int64_t)d * H + h) * kW + i] = c.win_log_a[((int64_t)s * H + h) * kW + i];
  for (int m = tid; m < M; m += kCopyThreads)
    if (j >> m & 1)
      c.page_log[(((int64_t)d * 2 + par) * M + m) * H + h] =
          c.page_log[(((int64_t)s * 2 + par) * M + m) * H + h];
  if (h == 0 && tid == 0) c.page_from[d * 2 + par] = c.page_from[s * 2 + par];
}

// ---------------------------------------------------------------- compact

// The i-th lowest free page below the number of pages in use takes the i-th lowest page in use
// above it; tables and counts follow here, the pages in cache_move_kernel.
__global__ void __launch_bounds__(kPlanThreads) cache_compact_plan_kernel(ll_cache c, int* n_live) {
  const Scratch sc = scratch_of(c);
  let_next_start();
  int live = 0;
  for (int64_t base = 0; base < c.n_pages; base += kPlanThreads) {
    const int64_t p = base + threadIdx.x;
    live += __syncthreads_count(p < c.n_pages && c.refcount[p] > 0);
  }
  int holes = 0, moves = 0;
  for (int64_t base = 0; base < c.n_pages; base += kPlanThreads) {
    const int64_t p = base + threadIdx.x;
    const bool used = p < c.n_pages && c.refcount[p] > 0;
    const bool hole = p < live && !used, move = p >= live && used;
    int n_hole, n_move;
    const int rank_h = holes + block_scan(hole, &n_hole);
    const int rank_m = moves + block_scan(move, &n_move);
    if (hole) sc.to[rank_h] = (int)p;
    if (move) sc.from[rank_m] = (int)p;
    holes += n_hole;
    moves += n_move;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < moves; i += kPlanThreads) {
    const int f = __ldcg(sc.from + i), t = __ldcg(sc.to + i);
    c.refcount[t] = c.refcount[f];
    c.refcount[f] = 0;
    sc.map[f] = t;
  }
  if (threadIdx.x == 0) {
    *sc.count = moves;
    *n_live = live;
  }
  if (moves == 0) return;
  __syncthreads();
  for (int64_t i = threadIdx.x; i < c.slots * c.levels; i += kPlanThreads) {
    const int e = c.page_table[i];
    if (e >= live && e < c.n_pages) c.page_table[i] = __ldcg(sc.map + e);
  }
}

// The moved pages, in chunks so that few pages fill the GPU too.  Bound by HBM: free, compact and
// two loads of 16 prompts of 16383 tokens take 200 us for 1.1 GB, 5.5 TB/s.
constexpr int kMoveChunk = 4 * kFlight * kCopyThreads;  // floats a CTA moves at a time

__global__ void __launch_bounds__(kCopyThreads) cache_move_kernel(ll_cache c) {
  const Scratch sc = scratch_of(c);
  wait_for_previous();
  const int64_t size = c.H * c.dk * c.dv, chunks = (size + kMoveChunk - 1) / kMoveChunk;
  const int64_t items = *sc.count * chunks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t i = it / chunks, o = (it - i * chunks) * kMoveChunk;
    const float* f = c.pages + sc.from[i] * size;
    float* t = c.pages + sc.to[i] * size;
    copy4(reinterpret_cast<float4*>(t + o), reinterpret_cast<const float4*>(f + o),
          min((int64_t)kMoveChunk, size - o) / 4, [](float4 x) { return x; });
  }
}

// CTAs per (row, head): doubled while that leaves the launch within the SMs, and each at least 16
// rows of the states.
int step_split(int64_t rows_heads, int dk, int sms) {
  int split = 1;
  while (split < kMaxSplit && rows_heads * split * 2 <= sms && dk >= 32 * split) split *= 2;
  return split;
}

}  // namespace

size_t cache_scratch_bytes(int64_t slots, int64_t n_pages) {
  return sizeof(int) * (size_t)(2 * slots + 3 * n_pages + 1);
}

cudaError_t launch_cache_reserve(const ll_cache& c, const int* slots, const int* pos, int64_t n,
                                 cudaStream_t s) {
  cache_reserve_kernel<<<1, kPlanThreads, 0, s>>>(c, slots, pos, n);
  return cudaGetLastError();
}

namespace {

template <typename T, typename OutT, bool kQueue>
cudaError_t launch_step(const ll_cache& c, StepArgs a, cudaStream_t s) {
  const size_t window = sizeof(T) * kW * (size_t)(c.dk + c.dv + 2 * kPad);
  // as many stages as leave room for two CTAs per SM (228 KB, 1 KB per CTA its own), at least two:
  // with fp32 tokens of dk = dv = 128 (window 68 KB) that is 256 bytes too many per CTA, and one runs
  a.stages = (int)std::max<size_t>(2, std::min<size_t>(kMaxStages, (115000 - sizeof(StepSmem) - window) / (kStageFloats * 4)));
  const size_t smem = window + (size_t)a.stages * kStageFloats * 4;
  const auto kernel = cache_step_kernel<T, OutT, kQueue>;
  const cudaError_t e = allow_shared(kernel);
  if (e != cudaSuccess) return e;
  // early only in the split form (8.3 -> 7.5 us with the reservation): in the queue's, CTAs that
  // find the reservation's still on their SM cost more than the launch (101 -> 104 us)
  return launch_following(!kQueue, kernel, dim3((unsigned)((int64_t)a.n * c.H * a.split)),
                          kQueue ? kQueueThreads : kSplitThreads, smem, a.split, s, c, a);
}

// The queue where there is more than an item for every SM, the split form below that.
template <typename T, typename OutT>
cudaError_t launch_form(const ll_cache& c, StepArgs a, cudaStream_t s) {
  const int64_t items = (int64_t)a.n * c.H;
  const int sms = sm_count();
  a.split = items > sms ? 1 : step_split(items, (int)c.dk, sms);
  return items > sms ? launch_step<T, OutT, true>(c, a, s) : launch_step<T, OutT, false>(c, a, s);
}

}  // namespace

cudaError_t launch_cache_step(const ll_cache& c, const int* slots, const int* pos, const void* q,
                              const void* k, const void* v, const float* log_a, const float* lam,
                              void* out, int n, int L, int out_dtype, cudaStream_t s) {
  StepArgs a;
  a.slots = slots; a.pos = pos; a.q = q; a.k = k; a.v = v; a.log_a = log_a; a.lam = lam;
  a.out = out; a.n = n; a.L = L; a.stages = 0;
  a.split = 1;
  const bool o32 = out_dtype == LL_F32;
  if (c.dtype == LL_F32)
    return o32 ? launch_form<float, float>(c, a, s) : launch_form<float, __nv_bfloat16>(c, a, s);
  return o32 ? launch_form<__nv_bfloat16, float>(c, a, s)
             : launch_form<__nv_bfloat16, __nv_bfloat16>(c, a, s);
}

cudaError_t launch_cache_load(const ll_cache& c, const int* slots, int64_t n, int T,
                              const float* state, int L, const void* k, const int64_t* sk,
                              const void* v, const int64_t* sv, const float* log_a,
                              const int64_t* sa, int Tk, cudaStream_t s) {
  cache_load_plan_kernel<<<1, kPlanThreads, 0, s>>>(c, slots, n, T);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || T == 0) return e;
  TokenStrides st;
  for (int i = 0; i < 3; ++i) {
    st.k[i] = sk[i];
    st.v[i] = sv[i];
    st.a[i] = sa[i];
  }
  int per = 0;
  for (int x = T >> kLogW; x; x &= x - 1) ++per;
  const dim3 grid((unsigned)(n * c.H), per + 1);
  if (c.dtype == LL_F32)
    return launch_following(true, cache_load_kernel<float>, grid, kCopyThreads, 0, 1, s, c, slots, T, state, L,
                            static_cast<const float*>(k), static_cast<const float*>(v), log_a, Tk, st);
  return launch_following(true, cache_load_kernel<__nv_bfloat16>, grid, kCopyThreads, 0, 1, s, c, slots, T, state,
                          L, static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v),
                          log_a, Tk, st);
}

cudaError_t launch_cache_store(const ll_cache& c, const int* slots, const int* pos, float* state,
                               int64_t n, int L, cudaStream_t s) {
  const dim3 grid((unsigned)(n * c.H), L);
  if (c.dtype == LL_F32) cache_store_kernel<float><<<grid, kCopyThreads, 0, s>>>(c, slots, pos, state, L);
  else cache_store_kernel<__nv_bfloat16><<<grid, kCopyThreads, 0, s>>>(c, slots, pos, state, L);
  return cudaGetLastError();
}

cudaError_t launch_cache_fork(const ll_cache& c, const int* src, const int* dst, const int* pos,
                              int64_t n, cudaStream_t s) {
  cache_fork_plan_kernel<<<1, kPlanThreads, 0, s>>>(c, src, dst, pos, n);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(n * c.H);
  return c.dtype == LL_F32
             ? launch_following(true, cache_fork_kernel<float>, dim3(grid), kCopyThreads, 0, 1, s, c, src, dst, pos)
             : launch_following(true, cache_fork_kernel<__nv_bfloat16>, dim3(grid), kCopyThreads, 0, 1, s, c, src,
                                dst, pos);
}

cudaError_t launch_cache_compact(const ll_cache& c, int* n_live, cudaStream_t s) {
  cache_compact_plan_kernel<<<1, kPlanThreads, 0, s>>>(c, n_live);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_following(true, cache_move_kernel, dim3(4 * sm_count()), kCopyThreads, 0, 1, s, c);
}

}  // namespace ll
