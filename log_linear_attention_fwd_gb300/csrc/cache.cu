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

#include "ll_internal.cuh"
#include "tc_ptx.cuh"

namespace ll {
namespace {

constexpr int kW = LL_CACHE_BLOCK;   // positions of a block
constexpr int kLogW = 6;             // log2(kW)
static_assert(kW == 1 << kLogW, "block length");

constexpr int kPlanThreads = 1024;
constexpr int kNone = 0x7fffffff;

// Scratch of the page operators: who owns each slot in this call, two lists and a map of pages.
struct Scratch {
  int* owner;  // [slots] lowest row of this call that names the slot
  int* from;   // [n_pages]
  int* to;     // [n_pages]
  int* map;    // [n_pages]
  int* count;  // [1]
};
__host__ __device__ Scratch scratch_of(const ll_cache& c) {
  Scratch s;
  s.owner = c.scratch;
  s.from = s.owner + c.slots;
  s.to = s.from + c.n_pages;
  s.map = s.to + c.n_pages;
  s.count = s.map + c.n_pages;
  return s;
}

__device__ __forceinline__ void raise(const ll_cache& c, unsigned bits) {
  atomicOr(c.error, bits);
}

// Sum of v over the threads before this one; *total over all.  kPlanThreads threads.
__device__ int block_scan(int v, int* total) {
  __shared__ int part[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // part may still be read from the call before
  if (lane == 31) part[w] = x;
  __syncthreads();
  if (w == 0) {
    int p = part[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, p, d);
      if (lane >= d) p += y;
    }
    part[lane] = p;
  }
  __syncthreads();
  *total = part[kPlanThreads / 32 - 1];
  return x - v + (w ? part[w - 1] : 0);
}

// Gives each named slot to the lowest row that names it.  Rows that name a slot out of range
// other than -1, or one that an earlier row has, raise the error word.
__device__ void claim_slots(const ll_cache& c, const int* slots, int64_t n, int* owner) {
  for (int64_t r = threadIdx.x; r < n; r += kPlanThreads) {
    const int s = slots[r];
    if (s >= 0 && s < c.slots) owner[s] = kNone;
  }
  __syncthreads();
  for (int64_t r = threadIdx.x; r < n; r += kPlanThreads) {
    const int s = slots[r];
    if (s >= 0 && s < c.slots) atomicMin(owner + s, (int)r);
    else if (s != -1) raise(c, LL_CACHE_ERR_SLOT);
  }
  __syncthreads();
  for (int64_t r = threadIdx.x; r < n; r += kPlanThreads) {
    const int s = slots[r];
    if (s >= 0 && s < c.slots && __ldcg(owner + s) != r) raise(c, LL_CACHE_ERR_SLOT);
  }
}
__device__ __forceinline__ bool owns(const ll_cache& c, const int* owner, int s, int64_t r) {
  return s >= 0 && s < c.slots && __ldcg(owner + s) == r;
}

__device__ __forceinline__ void drop_page(const ll_cache& c, int e) {
  if (e >= 0 && e < c.n_pages) atomicSub(c.refcount + e, 1);
}

// The last position a step can take: its block's fold still has a level to go to.
__device__ __forceinline__ bool position_ok(const ll_cache& c, int64_t t) {
  return t >= 0 && t < ((int64_t)kW << c.levels) - 1;
}

// Gives the lowest free pages to the table entries want[0..count), in that order.
__device__ void take_pages(const ll_cache& c, const int* want, int count) {
  int given = 0;
  for (int64_t base = 0; base < c.n_pages && given < count; base += kPlanThreads * 4) {
    const int64_t p0 = base + threadIdx.x * 4;
    int free_of[4], mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      free_of[i] = p0 + i < c.n_pages && __ldcg(c.refcount + p0 + i) == 0;
      mine += free_of[i];
    }
    int total, rank = given + block_scan(mine, &total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (free_of[i]) {
        if (rank < count) {
          c.page_table[__ldcg(want + rank)] = (int)(p0 + i);
          c.refcount[p0 + i] = 1;
        }
        ++rank;
      }
    given += total;
  }
  if (given < count && threadIdx.x == 0) raise(c, LL_CACHE_ERR_PAGES);
}

// ---------------------------------------------------------------- reserve, free

// reserve (pos given): each slot keeps the pages that are live at its position and, at a
// block's last position, has the page its fold goes to.  free (pos null): no page is kept.
__global__ void __launch_bounds__(kPlanThreads) cache_reserve_kernel(ll_cache c, const int* slots,
                                                                     const int* pos, int64_t n) {
  const Scratch sc = scratch_of(c);
  const int M = (int)c.levels;
  claim_slots(c, slots, n, sc.owner);
  for (int64_t k = threadIdx.x; k < n * M; k += kPlanThreads) {
    const int64_t r = k / M;
    const int m = (int)(k - r * M), s = slots[r];
    if (!owns(c, sc.owner, s, r)) continue;
    bool keep = false;
    if (pos) {
      const int t = pos[r];
      if (!position_ok(c, t)) {
        if (m == 0) raise(c, LL_CACHE_ERR_POSITION);
        continue;
      }
      const int j = t >> kLogW;
      keep = (j >> m) & 1 || ((t & (kW - 1)) == kW - 1 && m == __ffs(j + 1) - 1);
    }
    int* e = c.page_table + (int64_t)s * M + m;
    if (!keep && *e >= 0) {
      drop_page(c, *e);
      *e = -1;
    }
  }
  if (!pos) return;
  __syncthreads();
  int count = 0;
  for (int64_t base = 0; base < n; base += kPlanThreads) {
    const int64_t r = base + threadIdx.x;
    int at = -1;
    if (r < n && owns(c, sc.owner, slots[r], r) && position_ok(c, pos[r]) &&
        (pos[r] & (kW - 1)) == kW - 1) {
      const int64_t e = (int64_t)slots[r] * M + __ffs((pos[r] >> kLogW) + 1) - 1;
      if (c.page_table[e] < 0) at = (int)e;
    }
    int total;
    const int rank = count + block_scan(at >= 0, &total);
    if (at >= 0 && rank < c.n_pages) sc.from[rank] = at;
    count += total;
  }
  if (count == 0) return;
  __syncthreads();
  if (count > c.n_pages && threadIdx.x == 0) raise(c, LL_CACHE_ERR_PAGES);
  take_pages(c, sc.from, (int)min((int64_t)count, c.n_pages));
}

// ---------------------------------------------------------------- load

// The pages of n slots that hold T positions each.
__global__ void __launch_bounds__(kPlanThreads) cache_load_plan_kernel(ll_cache c,
                                                                       const int* slots,
                                                                       int64_t n, int64_t T) {
  const Scratch sc = scratch_of(c);
  const int M = (int)c.levels, j = (int)(T >> kLogW), per = __popc(j);
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

struct TokenStrides {
  int64_t k[3], v[3], a[3];  // batch, position, head
};

// blockIdx.y < per: one page of one (row, head) from the dense levels; the last: its tokens.
// T a multiple of 64: the block that ended with the prompt is folded, as the step at its last
// token would have: the levels that position T merges become the lowest page.
template <typename T_>
__global__ void __launch_bounds__(kCopyThreads) cache_load_kernel(
    ll_cache c, const int* __restrict__ slots, int T, const float* __restrict__ state, int L,
    const T_* __restrict__ k, const T_* __restrict__ v, const float* __restrict__ log_a, int Tk,
    TokenStrides st) {
  const int H = (int)c.H, G = (int)(c.H / c.Hqk), dk = (int)c.dk, dv = (int)c.dv;
  const int64_t row = blockIdx.x / H;
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
    for (int64_t i = threadIdx.x; i < n4; i += kCopyThreads) {
      float4 x = __ldcs(src + lo * n4 + i);
      for (int l = lo + 1; l <= hi; ++l) {
        const float4 y = __ldcs(src + l * n4 + i);
        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
      }
      dst[i] = x;
    }
    if (threadIdx.x == 0) c.page_log[(((int64_t)s * 2 + par) * M + m) * H + h] = 0.f;
    return;
  }
  if (h == 0 && threadIdx.x == 0) c.page_from[s * 2 + par] = r;
  const int t0 = Tk - r;  // the block's tokens are the last r given
  T_* wv = static_cast<T_*>(c.win_v) + ((int64_t)s * H + h) * kW * dv;
  for (int i = threadIdx.x; i < r * dv; i += kCopyThreads)
    wv[i] = v[row * st.v[0] + (t0 + i / dv) * st.v[1] + h * st.v[2] + i % dv];
  if (h % G == 0) {
    T_* wk = static_cast<T_*>(c.win_k) + ((int64_t)s * c.Hqk + h / G) * kW * dk;
    for (int i = threadIdx.x; i < r * dk; i += kCopyThreads)
      wk[i] = k[row * st.k[0] + (t0 + i / dk) * st.k[1] + (h / G) * st.k[2] + i % dk];
  }
  for (int i = threadIdx.x; i < r; i += kCopyThreads)
    c.win_log_a[((int64_t)s * H + h) * kW + i] =
        log_a ? log_a[row * st.a[0] + (t0 + i) * st.a[1] + h * st.a[2]] : 0.f;
}

// ---------------------------------------------------------------- decays inside a block

// after[i] = sum of la[u], i < u < r (0 at and past r - 1), and *since = sum of la[u], from <= u
// < r, for r <= 64 values.  One warp; sums run from the end, in one order.
__device__ __forceinline__ void block_decays(const float* la, int r, int from, float* after,
                                             float* since) {
  const int lane = threadIdx.x & 31;
  const float x0 = lane < r ? la[lane] : 0.f, x1 = lane + 32 < r ? la[lane + 32] : 0.f;
  float y0 = x0, y1 = x1;  // inclusive sums from the end of each half
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const float z0 = __shfl_down_sync(0xffffffffu, y0, d);
    const float z1 = __shfl_down_sync(0xffffffffu, y1, d);
    if (lane + d < 32) {
      y0 += z0;
      y1 += z1;
    }
  }
  const float upper = __shfl_sync(0xffffffffu, y1, 0);
  y0 += upper;
  float n0 = __shfl_down_sync(0xffffffffu, y0, 1), n1 = __shfl_down_sync(0xffffffffu, y1, 1);
  if (lane == 31) {
    n0 = upper;
    n1 = 0.f;
  }
  after[lane] = n0;
  after[lane + 32] = n1;
  const float f0 = __shfl_sync(0xffffffffu, y0, from & 31), f1 = __shfl_sync(0xffffffffu, y1, from & 31);
  if (lane == 0) *since = from >= r ? 0.f : from < 32 ? f0 : f1;
}

// ---------------------------------------------------------------- step

// A cluster of `split` CTAs per (row, head): each takes a share of the states' rows and of the block's
// tokens, and the first adds up their parts of the output (distributed shared memory).  Shares
// of rows are contiguous in a page; shares of columns were measured at twice the time for a
// single sequence, since each of their rows is a copy of its own.  A producer warp brings the
// tokens and then the pages, in stages of up to 16 KB, to shared memory by bulk copies; eight
// warps consume them.  Bound by HBM: a page of 128 x 128 is 64 KB for 32 KFLOP, and what counts
// is that copies are always in flight (two CTAs of four stages per SM).  A stage is kRowsPer
// rows per thread of one page; the pages of a row chunk come one after the other, so that a fold
// can sum them and the tokens' products for its rows in registers.
constexpr int kConsumers = 256;
constexpr int kStepThreads = kConsumers + 32;
constexpr int kStepWarps = kConsumers / 32;
constexpr int kRowsPer = 4;
constexpr int kStageFloats = kConsumers * 4 * kRowsPer;
constexpr int kMaxLevels = 24;
constexpr int kMaxSplit = 8;  // CTAs of a cluster

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 fma4(float s, float4 x, float4 y) {
  return make_float4(fmaf(s, x.x, y.x), fmaf(s, x.y, y.y), fmaf(s, x.z, y.z), fmaf(s, x.w, y.w));
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          tc::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float4 add4(float4 x, float4 y) {
  return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Writes v to p in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void store_remote4(float* p, uint32_t rank, float4 v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}

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

template <typename T, typename OutT>
__global__ void __launch_bounds__(kStepThreads, 2) cache_step_kernel(ll_cache c, StepArgs a) {
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ __align__(16) float vs[128], parts[kMaxSplit][128];
  __shared__ float4 red[kConsumers];
  __shared__ float qs[128], ks[128], lam[kMaxLevels + kLogW + 1], tok[kW], p[kW];
  __shared__ float page_e[kMaxLevels], since_s, self_s;
  __shared__ int page_at[kMaxLevels], page_lv[kMaxLevels], dest_s;
  __shared__ uint64_t full[8], empty[8], window;
  const int H = (int)c.H, G = (int)(c.H / c.Hqk), dk = (int)c.dk, dv = (int)c.dv;
  const int M = (int)c.levels, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int Z = a.split, sp = blockIdx.x % Z;  // the CTA's rank in its cluster
  const int64_t bh = blockIdx.x / Z, row = bh / H;
  const int h = (int)(bh - row * H), hq = h / G;
  const int s = a.slots[row], t = a.pos[row];
  if (s == -1) return;
  // rows with a slot that is out of range, given to an earlier row, or at a position outside the
  // cache are left as they are
  unsigned bad = s < 0 || s >= c.slots ? LL_CACHE_ERR_SLOT : 0;
  if (!bad && !position_ok(c, t)) bad = LL_CACHE_ERR_POSITION;
  if (bad) {
    if (tid == 0 && sp == 0 && h == 0) raise(c, bad);
    return;
  }
  const int j = t >> kLogW, r = t & (kW - 1), par = j & 1;
  const bool fold = r == kW - 1;
  const int to = fold ? __ffs(j + 1) - 1 : -1;  // the level the block is folded to
  const int live = __popc(j);
  // this CTA's state rows [k0, k1) and tokens [t0, t1); a fold needs all tokens' products, so it
  // brings them all
  const int share = (dk + Z - 1) / Z, k0 = min(dk, sp * share), k1 = min(dk, k0 + share);
  const int tokens = ((r + Z - 1) / Z + 7) & ~7, t0 = min(r, sp * tokens), t1 = min(r, t0 + tokens);
  const int b0 = fold ? 0 : t0, b1 = fold ? r : t1;  // tokens to bring
  const int groups = dv >> 2, lanes = kConsumers / groups;       // column groups, threads down the rows
  const int per = min(kRowsPer, (share + lanes - 1) / lanes);    // rows of a thread in a stage
  const int span = per * lanes, chunks = (k1 - k0 + span - 1) / span;
  float* ring = reinterpret_cast<float*>(dyn);
  T* wks = reinterpret_cast<T*>(dyn + (size_t)a.stages * kStageFloats * 4);
  T* wvs = wks + kW * dk;
  const T* k = static_cast<const T*>(a.k) + (row * c.Hqk + hq) * dk;
  const T* v = static_cast<const T*>(a.v) + bh * dv;
  const float la = a.log_a ? a.log_a[bh] : 0.f;
  bool ok = true;
  if (w == kStepWarps) {  // the producer
    if (lane == 0) {
      for (int i = 0; i < a.stages; ++i) {
        tc::mbar_init(&full[i], 1);
        tc::mbar_init(&empty[i], kStepWarps);
      }
      tc::mbar_init(&window, 1);
      tc::fence_mbar_init();
      if (b1 > b0) {
        // whole rows from a multiple of 8 rows on: 16-byte aligned; the length is rounded up to
        // 16 bytes, still inside the window
        const int64_t ok0 = (((int64_t)s * c.Hqk + hq) * kW + b0) * dk;
        const int64_t ov0 = (((int64_t)s * H + h) * kW + b0) * dv;
        const uint32_t nk = ((b1 - b0) * dk * sizeof(T) + 15) & ~15u;
        const uint32_t nv = ((b1 - b0) * dv * sizeof(T) + 15) & ~15u;
        tc::mbar_arrive_expect_tx(&window, nk + nv);
        bulk_load(wks + b0 * dk, static_cast<const T*>(c.win_k) + ok0, nk, &window);
        bulk_load(wvs + b0 * dv, static_cast<const T*>(c.win_v) + ov0, nv, &window);
      }
    }
    __syncwarp();
    // the live pages, lowest level first
    const bool here = lane < M && (j >> lane) & 1;
    int e = 0;
    if (here || lane == to) {
      e = c.page_table[(int64_t)s * M + lane];
      if (e < 0 || e >= c.n_pages) ok = false;
    }
    if (here) {
      const int at = __popc(j & ((1 << lane) - 1));
      page_at[at] = e;
      page_lv[at] = lane;
    }
    if (lane == to) dest_s = e;
  } else {
    if (w == 0) {
      block_decays(c.win_log_a + ((int64_t)s * H + h) * kW, r, c.page_from[s * 2 + par], tok, &since_s);
      const bool here = lane < M && (j >> lane) & 1;
      const float log = here ? c.page_log[(((int64_t)s * 2 + par) * M + lane) * H + h] : 0.f;
      __syncwarp();
      if (here) page_e[__popc(j & ((1 << lane) - 1))] = log + since_s + la;
      for (int i = lane; i < kW; i += 32) tok[i] = expf(tok[i] + la);
    }
    const T* q = static_cast<const T*>(a.q) + (row * c.Hqk + hq) * dk;
    for (int i = tid; i < dk; i += kConsumers) {
      qs[i] = to_f32(q[i]);
      ks[i] = to_f32(k[i]);
    }
    for (int i = tid; i < dv; i += kConsumers) vs[i] = to_f32(v[i]);
    for (int i = tid; i < M + kLogW + 1; i += kConsumers) lam[i] = a.lam[bh * a.L + i];
    for (int64_t i = tid; i < row; i += kConsumers)
      if (a.slots[i] == s) bad = LL_CACHE_ERR_SLOT;
  }
  const bool twice = __syncthreads_or(bad != 0);
  const bool missing = !__syncthreads_and(ok);
  if (twice || missing) {  // the same for the whole cluster
    if (tid == 0 && sp == 0 && h == 0) raise(c, twice ? LL_CACHE_ERR_SLOT : LL_CACHE_ERR_MISSING);
    if (w == kStepWarps && b1 > b0) tc::mbar_wait(&window, 0);  // its copies end before the CTA does
    return;
  }
  if (Z > 1) cluster_arrive();  // this CTA is there
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (w == kStepWarps) {
    int st = 0, phase = 0;
    for (int ck = 0; ck < chunks && lane == 0; ++ck) {
      const int d0 = k0 + ck * span, bytes = min(span, k1 - d0) * dv * 4;
      for (int m = 0; m < live; ++m) {
        ok = tc::mbar_wait(&empty[st], phase ^ 1) && ok;
        tc::mbar_arrive_expect_tx(&full[st], bytes);
        bulk_load(ring + st * kStageFloats, c.pages + (((int64_t)page_at[m] * H + h) * dk + d0) * dv,
                  bytes, &full[st]);
        if (++st == a.stages) {
          st = 0;
          phase ^= 1;
        }
      }
    }
  } else {
    // scores of the CTA's tokens: a warp takes every eighth; the first CTA has the new one too
    if (b1 > b0) ok = tc::mbar_wait(&window, 0);
    for (int i = t0 + w; i < t1; i += kStepWarps) {
      float x = 0.f;
      for (int d = lane; d < dk; d += 32) x = fmaf(qs[d], to_f32(wks[i * dk + d]), x);
#pragma unroll
      for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      if (lane == 0) p[i] = lam[fenwick_level(r, i)] * tok[i] * x;
    }
    if (sp == 0 && w == 0) {
      float x = 0.f;
      for (int d = lane; d < dk; d += 32) x = fmaf(qs[d], ks[d], x);
#pragma unroll
      for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      if (lane == 0) self_s = lam[0] * x;
    }
    const int cg = tid % groups, row0 = tid / groups;
    const bool on = row0 < lanes;
    asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
    const float4 v4 = *reinterpret_cast<const float4*>(vs + 4 * cg);
    if (on) {
      if (row0 == 0 && sp == 0) acc = fma4(self_s, v4, acc);
      for (int i = t0 + row0; i < t1; i += lanes) acc = fma4(p[i], load4(wvs + i * dv + 4 * cg), acc);
    }
    int st = 0, phase = 0;
    for (int ck = 0; ck < chunks; ++ck) {
      const int d0 = k0 + ck * span + per * row0;
      const int n = on ? min(per, k1 - d0) : 0;  // this thread's rows (below 1: none)
      float qr[kRowsPer];
      float4 sum[kRowsPer];
#pragma unroll
      for (int x = 0; x < kRowsPer; ++x) {
        qr[x] = x < n ? qs[d0 + x] : 0.f;
        sum[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      for (int m = 0; m < live; ++m) {
        ok = tc::mbar_wait(&full[st], phase) && ok;
        const float* P = ring + st * kStageFloats + per * row0 * dv + 4 * cg;
        const float e = expf(page_e[m]);
        float4 part = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < kRowsPer; ++x)
          if (x < n) {
            const float4 y = *reinterpret_cast<const float4*>(P + x * dv);
            part = fma4(qr[x], y, part);
            if (page_lv[m] < to) sum[x] = fma4(e, y, sum[x]);
          }
        acc = fma4(e * lam[kLogW + 1 + page_lv[m]], part, acc);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&empty[st]);
        if (++st == a.stages) {
          st = 0;
          phase ^= 1;
        }
      }
      if (fold && n > 0) {
        for (int i = 0; i < r; ++i) {
          const float4 y = load4(wvs + i * dv + 4 * cg);
          const float e = tok[i];
#pragma unroll
          for (int x = 0; x < kRowsPer; ++x)
            if (x < n) sum[x] = fma4(e * to_f32(wks[i * dk + d0 + x]), y, sum[x]);
        }
        if (ok) {
          float* D = c.pages + (((int64_t)dest_s * H + h) * dk + d0) * dv + 4 * cg;
#pragma unroll
          for (int x = 0; x < kRowsPer; ++x)
            if (x < n) *reinterpret_cast<float4*>(D + x * dv) = fma4(ks[d0 + x], v4, sum[x]);
        }
      }
    }
    red[tid] = acc;
    if (!ok) raise(c, LL_CACHE_ERR_WAIT);
    asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
    if (tid < groups) {
      acc = red[tid];
      for (int i = 1; i < lanes; ++i) acc = add4(acc, red[tid + i * groups]);
    }
  }
  if (Z > 1) {
    __syncwarp();
    cluster_wait();  // all CTAs are there
    if (tid < groups) store_remote4(&parts[sp][4 * tid], 0, acc);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (sp == 0 && tid < groups) {
      acc = *reinterpret_cast<const float4*>(&parts[0][4 * tid]);
      for (int z = 1; z < Z; ++z) acc = add4(acc, *reinterpret_cast<const float4*>(&parts[z][4 * tid]));
    }
  }
  if (sp == 0 && tid < groups) {
    OutT* o = static_cast<OutT*>(a.out) + bh * dv + 4 * tid;
    o[0] = from_f32<OutT>(acc.x);
    o[1] = from_f32<OutT>(acc.y);
    o[2] = from_f32<OutT>(acc.z);
    o[3] = from_f32<OutT>(acc.w);
  }
  // this token joins the block
  if (sp == Z - 1) {
    for (int i = tid; i < dv; i += kStepThreads)
      static_cast<T*>(c.win_v)[(((int64_t)s * H + h) * kW + r) * dv + i] = v[i];
    if (h % G == 0)
      for (int i = tid; i < dk; i += kStepThreads)
        static_cast<T*>(c.win_k)[(((int64_t)s * c.Hqk + hq) * kW + r) * dk + i] = k[i];
    if (tid == 0) c.win_log_a[((int64_t)s * H + h) * kW + r] = la;
    if (fold) {  // what the next block's steps read
      if (tid < live && page_lv[tid] > to)
        c.page_log[(((int64_t)s * 2 + (par ^ 1)) * M + page_lv[tid]) * H + h] = page_e[tid];
      if (tid == 0) {
        c.page_log[(((int64_t)s * 2 + (par ^ 1)) * M + to) * H + h] = 0.f;
        if (h == 0) c.page_from[s * 2 + (par ^ 1)] = 0;
      }
    }
  }
}

// ---------------------------------------------------------------- store

// One CTA per (row, head, level): the dense state's level, from a page or from the tokens.
template <typename T>
__global__ void __launch_bounds__(kCopyThreads) cache_store_kernel(
    ll_cache c, const int* __restrict__ slots, const int* __restrict__ pos,
    float* __restrict__ state, int L) {
  __shared__ float tok[kW], since_s, es[kW];
  const int H = (int)c.H, G = (int)(c.H / c.Hqk), dk = (int)c.dk, dv = (int)c.dv;
  const int M = (int)c.levels, tid = threadIdx.x, level = blockIdx.y;
  const int64_t row = blockIdx.x / H;
  const int h = (int)(blockIdx.x - row * H), s = slots[row], n = pos[row];
  if (s == -1) return;
  unsigned bad = s < 0 || s >= c.slots ? LL_CACHE_ERR_SLOT : 0;
  if (!bad && (n < 0 || n > ((int64_t)kW << M) - 1)) bad = LL_CACHE_ERR_POSITION;
  if (bad) {
    if (tid == 0 && h == 0 && level == 0) raise(c, bad);
    return;
  }
  const int j = n >> kLogW, r = n & (kW - 1), par = j & 1;
  if (tid < 32)
    block_decays(c.win_log_a + ((int64_t)s * H + h) * kW, r, c.page_from[s * 2 + par], tok, &since_s);
  __syncthreads();
  const int64_t size = (int64_t)dk * dv, n4 = size / 4;
  float4* dst = reinterpret_cast<float4*>(state + ((row * H + h) * (int64_t)L + level) * size);
  // a page i is level 7 + i; after a whole block the lowest one holds the sum of the levels that
  // the next step merges, and stands in the highest of them
  const int low = r == 0 && j ? __ffs(j) - 1 : -1;
  const int m = low >= 0 && level == kLogW + low ? low : level - kLogW - 1;
  if (m >= 0 && m < M && (j >> m & 1) && !(m == low && level != kLogW + low)) {
    const int e = c.page_table[(int64_t)s * M + m];
    if (e < 0 || e >= c.n_pages) {
      if (tid == 0) raise(c, LL_CACHE_ERR_MISSING);
      return;
    }
    const float f = expf(c.page_log[(((int64_t)s * 2 + par) * M + m) * H + h] + since_s);
    const float4* src = reinterpret_cast<const float4*>(c.pages + ((int64_t)e * H + h) * size);
    for (int64_t i = tid; i < n4; i += kCopyThreads) {
      const float4 x = __ldcs(src + i);
      __stcs(dst + i, make_float4(f * x.x, f * x.y, f * x.z, f * x.w));
    }
    return;
  }
  // tokens lo .. hi - 1 of the block, as seen from its last one
  int lo = 0, hi = 0;
  if (r > 0 && level <= kLogW) {
    const int last = r - 1;
    if (level == 0) {
      lo = last;
      hi = r;
    } else if (last >> (level - 1) & 1) {
      lo = ((last >> (level - 1)) - 1) << (level - 1);
      hi = lo + (1 << (level - 1));
    }
  }
  for (int i = lo + tid; i < hi; i += kCopyThreads) es[i] = expf(tok[i]);
  __syncthreads();
  const T* wk = static_cast<const T*>(c.win_k) + ((int64_t)s * c.Hqk + h / G) * kW * dk;
  const T* wv = static_cast<const T*>(c.win_v) + ((int64_t)s * H + h) * kW * dv;
  for (int64_t i = tid; i < n4; i += kCopyThreads) {
    const int d = (int)(4 * i / dv), col = (int)(4 * i - (int64_t)d * dv);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int u = lo; u < hi; ++u)
      x = fma4(es[u] * to_f32(wk[u * dk + d]), load4(wv + u * dv + col), x);
    __stcs(dst + i, x);
  }
}

// ---------------------------------------------------------------- fork

// A row is left out where its target is not its own, its source is not a slot or is some row's
// target, or its position is outside the cache.  owner: the targets' rows, kNone for sources.
__device__ __forceinline__ unsigned fork_bad(const ll_cache& c, const int* owner, int s, int t) {
  if (s < 0 || s >= c.slots || __ldcg(owner + s) != kNone) return LL_CACHE_ERR_SLOT;
  return t < 0 || t > ((int64_t)kW << c.levels) - 1 ? LL_CACHE_ERR_POSITION : 0;
}

__global__ void __launch_bounds__(kPlanThreads) cache_fork_plan_kernel(ll_cache c, const int* src,
                                                                       const int* dst,
                                                                       const int* pos, int64_t n) {
  const Scratch sc = scratch_of(c);
  const int M = (int)c.levels;
  for (int64_t r = threadIdx.x; r < n; r += kPlanThreads)
    if (src[r] >= 0 && src[r] < c.slots) sc.owner[src[r]] = kNone;
  __syncthreads();
  claim_slots(c, dst, n, sc.owner);
  // first every target gives up its pages, then it takes a share of its source's
  for (int take = 0; take < 2; ++take) {
    for (int64_t k = threadIdx.x; k < n * M; k += kPlanThreads) {
      const int64_t r = k / M;
      const int m = (int)(k - r * M), s = src[r], d = dst[r], t = pos[r];
      if (!owns(c, sc.owner, d, r)) continue;
      const unsigned bad = fork_bad(c, sc.owner, s, t);
      if (bad) {
        if (m == 0 && !take) raise(c, bad);
        continue;
      }
      int* e = c.page_table + (int64_t)d * M + m;
      if (!take) {
        if (*e >= 0) drop_page(c, *e);
        *e = -1;
      } else if ((t >> kLogW) >> m & 1) {
        const int page = c.page_table[(int64_t)s * M + m];
        if (page < 0 || page >= c.n_pages) {
          raise(c, LL_CACHE_ERR_MISSING);
        } else {
          atomicAdd(c.refcount + page, 1);
          *e = page;
        }
      }
    }
    __syncthreads();
  }
}

// One CTA per (row, head): the tokens of the source's block, and its pages' decays.
template <typename T>
__global__ void __launch_bounds__(kCopyThreads) cache_fork_kernel(ll_cache c,
                                                                  const int* __restrict__ src,
                                                                  const int* __restrict__ dst,
                                                                  const int* __restrict__ pos) {
  const int H = (int)c.H, G = (int)(c.H / c.Hqk), dk = (int)c.dk, dv = (int)c.dv;
  const int M = (int)c.levels, tid = threadIdx.x;
  const int64_t row = blockIdx.x / H;
  const int h = (int)(blockIdx.x - row * H), s = src[row], d = dst[row], t = pos[row];
  const int* owner = scratch_of(c).owner;
  if (!owns(c, owner, d, row) || fork_bad(c, owner, s, t)) return;
  const int j = t >> kLogW, r = t & (kW - 1), par = j & 1;
  const T* fv = static_cast<const T*>(c.win_v) + ((int64_t)s * H + h) * kW * dv;
  T* tv = static_cast<T*>(c.win_v) + ((int64_t)d * H + h) * kW * dv;
  for (int i = tid; i < r * dv; i += kCopyThreads) tv[i] = fv[i];
  if (h % G == 0) {
    const T* fk = static_cast<const T*>(c.win_k) + ((int64_t)s * c.Hqk + h / G) * kW * dk;
    T* tk = static_cast<T*>(c.win_k) + ((int64_t)d * c.Hqk + h / G) * kW * dk;
    for (int i = tid; i < r * dk; i += kCopyThreads) tk[i] = fk[i];
  }
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

constexpr int kMoveChunk = 16 * kCopyThreads;  // floats a CTA moves at a time

__global__ void __launch_bounds__(kCopyThreads) cache_move_kernel(ll_cache c) {
  const Scratch sc = scratch_of(c);
  const int64_t size = c.H * c.dk * c.dv, chunks = (size + kMoveChunk - 1) / kMoveChunk;
  const int64_t items = *sc.count * chunks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t i = it / chunks, o = (it - i * chunks) * kMoveChunk;
    const float* f = c.pages + sc.from[i] * size;
    float* t = c.pages + sc.to[i] * size;
    float4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t at = o + 4 * (u * kCopyThreads + threadIdx.x);
      if (at < size) x[u] = __ldcs(reinterpret_cast<const float4*>(f + at));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t at = o + 4 * (u * kCopyThreads + threadIdx.x);
      if (at < size) __stcs(reinterpret_cast<float4*>(t + at), x[u]);
    }
  }
}

// CTAs per (row, head): doubled while that leaves the launch within two CTAs per SM, and each at
// least 16 rows of the states.
int step_split(int64_t rows_heads, int dk) {
  int split = 1;
  while (split < kMaxSplit && rows_heads * split * 2 <= 2 * 152 && dk >= 32 * split) split *= 2;
  return split;
}

}  // namespace

size_t cache_scratch_bytes(int64_t slots, int64_t n_pages) {
  return sizeof(int) * (size_t)(slots + 3 * n_pages + 1);
}

cudaError_t launch_cache_reserve(const ll_cache& c, const int* slots, const int* pos, int64_t n,
                                 cudaStream_t s) {
  cache_reserve_kernel<<<1, kPlanThreads, 0, s>>>(c, slots, pos, n);
  return cudaGetLastError();
}

namespace {

template <typename T, typename OutT>
cudaError_t launch_step(const ll_cache& c, StepArgs a, cudaStream_t s) {
  const size_t window = sizeof(T) * kW * (size_t)(c.dk + c.dv);
  // as many stages as leave room for two CTAs per SM (and at least two); 12 KB are static
  a.stages = (int)std::max<size_t>(2, std::min<size_t>(8, (100 * 1024 - window) / (kStageFloats * 4)));
  const size_t smem = window + (size_t)a.stages * kStageFloats * 4;
  const cudaError_t e = cudaFuncSetAttribute(cache_step_kernel<T, OutT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.n * c.H * a.split));
  cfg.blockDim = dim3(kStepThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = a.split;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, cache_step_kernel<T, OutT>, c, a);
}

}  // namespace

cudaError_t launch_cache_step(const ll_cache& c, const int* slots, const int* pos, const void* q,
                              const void* k, const void* v, const float* log_a, const float* lam,
                              void* out, int n, int L, int out_dtype, cudaStream_t s) {
  StepArgs a;
  a.slots = slots; a.pos = pos; a.q = q; a.k = k; a.v = v; a.log_a = log_a; a.lam = lam;
  a.out = out; a.n = n; a.L = L; a.stages = 0;
  a.split = step_split((int64_t)n * c.H, (int)c.dk);
  const bool o32 = out_dtype == LL_F32;
  if (c.dtype == LL_F32)
    return o32 ? launch_step<float, float>(c, a, s) : launch_step<float, __nv_bfloat16>(c, a, s);
  return o32 ? launch_step<__nv_bfloat16, float>(c, a, s)
             : launch_step<__nv_bfloat16, __nv_bfloat16>(c, a, s);
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
    cache_load_kernel<float><<<grid, kCopyThreads, 0, s>>>(
        c, slots, T, state, L, static_cast<const float*>(k), static_cast<const float*>(v), log_a,
        Tk, st);
  else
    cache_load_kernel<__nv_bfloat16><<<grid, kCopyThreads, 0, s>>>(
        c, slots, T, state, L, static_cast<const __nv_bfloat16*>(k),
        static_cast<const __nv_bfloat16*>(v), log_a, Tk, st);
  return cudaGetLastError();
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
  if (c.dtype == LL_F32) cache_fork_kernel<float><<<grid, kCopyThreads, 0, s>>>(c, src, dst, pos);
  else cache_fork_kernel<__nv_bfloat16><<<grid, kCopyThreads, 0, s>>>(c, src, dst, pos);
  return cudaGetLastError();
}

cudaError_t launch_cache_compact(const ll_cache& c, int* n_live, cudaStream_t s) {
  cache_compact_plan_kernel<<<1, kPlanThreads, 0, s>>>(c, n_live);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cache_move_kernel<<<152 * 4, kCopyThreads, 0, s>>>(c);
  return cudaGetLastError();
}

}  // namespace ll
