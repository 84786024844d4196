// What the operators on the paged decode cache share: its layout, the claiming of slots and pages,
// decays inside a block, and small copies and products.
#pragma once

#include "ll_internal.cuh"
#include "tc_ptx.cuh"

namespace ll {

constexpr int kW = LL_CACHE_BLOCK;   // positions of a block
constexpr int kLogW = 6;             // log2(kW)
static_assert(kW == 1 << kLogW, "block length");

constexpr int kMaxLevels = 24;

constexpr int kPlanThreads = 1024;
constexpr int kNone = 0x7fffffff;

// Scratch of the page operators: who owns each slot in this call, two lists and a map of pages.
struct Scratch {
  int* owner;  // [slots] lowest row of this call that names the slot
  int* done;   // [slots] CTAs that have read the slot's block
  int* from;   // [n_pages]
  int* to;     // [n_pages]
  int* map;    // [n_pages]
  int* count;  // [1]
};
__host__ __device__ __forceinline__ Scratch scratch_of(const ll_cache& c) {
  Scratch s;
  s.owner = c.scratch;
  s.done = s.owner + c.slots;
  s.from = s.done + c.slots;
  s.to = s.from + c.n_pages;
  s.map = s.to + c.n_pages;
  s.count = s.map + c.n_pages;
  return s;
}

// The page operators are a small kernel that settles the tables and a large one that follows it;
// the second is launched while the first runs (programmatic dependent launch), and waits for
// its end before it touches memory: that hides the launch, 1 to 2 us.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_following(bool early, void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                             int cluster, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = early;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

__device__ __forceinline__ void raise(const ll_cache& c, unsigned bits) {
  atomicOr(c.error, bits);
}

// Sum of v over the threads before this one; *total over all.  kPlanThreads threads.
inline __device__ int block_scan(int v, int* total) {
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
// other than -1, or one that an earlier row has, raise the error word.  src: rows with -1 there
// name none.
inline __device__ void claim_slots(const ll_cache& c, const int* slots, int64_t n, int* owner,
                            const int* src = nullptr) {
  auto slot_of = [&](int64_t r) { return src && src[r] == -1 ? -1 : slots[r]; };
  for (int64_t r = threadIdx.x; r < n; r += kPlanThreads) {
    const int s = slot_of(r);
    if (s >= 0 && s < c.slots) owner[s] = kNone;
  }
  __syncthreads();
  for (int64_t r = threadIdx.x; r < n; r += kPlanThreads) {
    const int s = slot_of(r);
    if (s >= 0 && s < c.slots) atomicMin(owner + s, (int)r);
    else if (s != -1) raise(c, LL_CACHE_ERR_SLOT);
  }
  __syncthreads();
  for (int64_t r = threadIdx.x; r < n; r += kPlanThreads) {
    const int s = slot_of(r);
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

// Whether a slot's pages, if it has any at n positions, have already decayed past there: a prompt
// was loaded up to a later position of the block.
__device__ __forceinline__ bool before_pages(const ll_cache& c, int s, int n) {
  const int j = n >> kLogW;
  return j && c.page_from[s * 2 + (j & 1)] > (n & (kW - 1));
}

// Gives the lowest free pages to the table entries want[0..count), in that order.
inline __device__ void take_pages(const ll_cache& c, const int* want, int count) {
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
          c.page_table[want[rank]] = (int)(p0 + i);
          c.refcount[p0 + i] = 1;
        }
        ++rank;
      }
    given += total;
  }
  if (given < count && threadIdx.x == 0) raise(c, LL_CACHE_ERR_PAGES);
}

// The pages of n rows: slot_of(r) (-1: the row is left out) keeps those that are live in block
// block_of(r) and, where fold_of(r), has the page that the block is folded to.  That page is the
// slot's alone: one that is left over from earlier positions and shared is given up like the
// others.  One CTA of kPlanThreads: the order of the rows decides who gets which page.
template <typename SlotOf, typename BlockOf, typename FoldOf>
__device__ __forceinline__ void settle_pages(const ll_cache& c, int64_t n, SlotOf slot_of, BlockOf block_of,
                                             FoldOf fold_of) {
  const Scratch sc = scratch_of(c);
  const int M = (int)c.levels, tid = threadIdx.x;
  bool folds = false;
  for (int64_t r = tid; r < n; r += kPlanThreads) folds |= slot_of(r) >= 0 && fold_of(r);
  folds = __syncthreads_or(folds);
  if (folds) {  // mark shared pages where folds go to, before any count changes: -2 - page
    for (int64_t r = tid; r < n; r += kPlanThreads) {
      const int s = slot_of(r);
      if (s < 0 || !fold_of(r)) continue;
      int* e = c.page_table + (int64_t)s * M + __ffs(block_of(r) + 1) - 1;
      if (*e < 0 || *e >= c.n_pages) *e = -1;  // (a table that was overwritten: no page, and no mark)
      else if (__ldcg(c.refcount + *e) != 1) *e = -2 - *e;
    }
    __syncthreads();
  }
  for (int64_t k = tid; k < n * M; k += kPlanThreads) {
    const int64_t r = k / M;
    const int m = (int)(k - r * M), s = slot_of(r);
    if (s < 0) continue;
    const int j = block_of(r);
    const bool to = fold_of(r) && m == __ffs(j + 1) - 1;
    const bool keep = to || (j >> m) & 1;
    int* e = c.page_table + (int64_t)s * M + m;
    if (*e < -1 || (!keep && *e >= 0)) {
      drop_page(c, to ? -2 - *e : *e);  // (below -1 elsewhere: no page)
      *e = -1;
    }
  }
  if (!folds) return;
  __syncthreads();
  int count = 0;
  for (int64_t base = 0; base < n; base += kPlanThreads) {
    const int64_t r = base + tid;
    int at = -1;
    if (r < n && slot_of(r) >= 0 && fold_of(r)) {
      const int64_t e = (int64_t)slot_of(r) * M + __ffs(block_of(r) + 1) - 1;
      if (c.page_table[e] < 0) at = (int)e;
    }
    int total;
    const int rank = count + block_scan(at >= 0, &total);
    if (at >= 0 && rank < c.n_pages) sc.from[rank] = at;
    count += total;
  }
  if (count == 0) return;
  __syncthreads();
  if (count > c.n_pages && tid == 0) raise(c, LL_CACHE_ERR_PAGES);
  take_pages(c, sc.from, (int)min((int64_t)count, c.n_pages));
}

// The table's entry for the page that slot s folds block j to (-1: none), and whether that page is shared.
__device__ __forceinline__ int fold_page(const ll_cache& c, int s, int j, bool* shared) {
  const int e = c.page_table[(int64_t)s * c.levels + __ffs(j + 1) - 1];
  const bool page = e >= 0 && e < c.n_pages;
  *shared = page && __ldcg(c.refcount + e) != 1;
  return page ? e : -1;
}

// settle_pages for up to kPlanThreads rows, thread r having row r: its slot (-1: left out), block j and, where the
// block is folded, what fold_page gives before any of this.  Spares the general form's marks and lists in memory and
// the reads behind them (reservation and step of 128 rows 101.9 -> 100.3 us).
__device__ __forceinline__ void settle_few(const ll_cache& c, int n, int s, int j, bool fold, int e, bool shared) {
  __shared__ int slot_s[kPlanThreads], block_s[kPlanThreads], want[kPlanThreads];
  const int M = (int)c.levels, tid = threadIdx.x, at = s * M + __ffs(j + 1) - 1;
  fold &= s >= 0;
  const bool need = fold && (e < 0 || shared);
  slot_s[tid] = s;
  block_s[tid] = fold ? ~j : j;
  const bool folds = __syncthreads_or(fold);
  for (int k = tid; k < n * M; k += kPlanThreads) {
    const int r = k / M, m = k - r * M, b = block_s[r], jr = b < 0 ? ~b : b;
    if (slot_s[r] < 0 || (b < 0 && m == __ffs(jr + 1) - 1)) continue;
    int* p = c.page_table + slot_s[r] * M + m;
    const int x = *p;
    if (x < -1 || (x >= 0 && !(jr >> m & 1))) {
      drop_page(c, x);
      *p = -1;
    }
  }
  if (need) {
    if (shared) drop_page(c, e);
    c.page_table[at] = -1;
  }
  if (!folds) return;
  int total;
  const int rank = block_scan(need, &total);
  if (need) want[rank] = at;
  if (total == 0) return;
  __syncthreads();
  take_pages(c, want, total);
}

// ---------------------------------------------------------------- decays inside a block

// after[i] = sum of la[u], i < u < r (0 at and past r - 1), and *since = sum of la[u], from <= u
// < r, for r <= 64 values.  One warp; sums run from the end, in one order.
__device__ __forceinline__ void block_decays(float x0, float x1, int r, int from, float* after,
                                             float* since) {
  const int lane = threadIdx.x & 31;  // x0, x1: la[lane] and la[lane + 32], 0 from r on
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
  *since = from >= r ? 0.f : from < 32 ? f0 : f1;
}

__device__ __forceinline__ void block_decays(const float* la, int r, int from, float* after,
                                             float* since) {  // *since in every lane
  const int lane = threadIdx.x & 31;
  block_decays(lane < r ? la[lane] : 0.f, lane + 32 < r ? la[lane + 32] : 0.f, r, from, after, since);
}

// ---------------------------------------------------------------- vectors, copies, clusters

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

template <typename OutT>
__device__ __forceinline__ void store_out(void* out, int64_t at, float4 v) {
  OutT* o = static_cast<OutT*>(out) + at;
  o[0] = from_f32<OutT>(v.x);
  o[1] = from_f32<OutT>(v.y);
  o[2] = from_f32<OutT>(v.z);
  o[3] = from_f32<OutT>(v.w);
}

// Why a row cannot be served, before its pages are looked at.
__device__ __forceinline__ unsigned row_bad(const ll_cache& c, int s, int t) {
  if (s < 0 || s >= c.slots) return LL_CACHE_ERR_SLOT;
  return position_ok(c, t) ? 0 : LL_CACHE_ERR_POSITION;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
// ---------------------------------------------------------------- tensor cores

__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], const __nv_bfloat16* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(tc::smem_u32(p))
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x's leading bf16 parts (x >= 0); x keeps the rest, at least `least`.
__device__ __forceinline__ uint32_t take_bf16(float2& x, float2 least) {
  uint32_t h;
  asm("cvt.rz.bf16x2.f32 %0, %2, %1;" : "=r"(h) : "f"(x.x), "f"(x.y));
  const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h));
  x = make_float2(fmaxf(x.x - f.x, least.x), fmaxf(x.y - f.y, least.y));
  return h;
}
// The B fragments of a fold: 8 columns of the block's 64 values, decayed, as three bf16 parts which together are
// the fp32 product; infinities as take_bf16 keeps them.  wvs: [token][vp], tok: the tokens' decays.
__device__ __forceinline__ void load_decayed(uint32_t (&b)[kW / 16][3][2], const __nv_bfloat16* wvs, const float* tok,
                                             int vp) {
  const int lane = threadIdx.x & 31, i = 2 * (lane & 3);
#pragma unroll
  for (int ks = 0; ks < kW / 16; ks += 2) {
    uint32_t r[4];  // tokens 16 ks .. + 31 of 8 columns
    ldmatrix_trans(r, wvs + (16 * ks + lane) * vp);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = 16 * ks + 8 * u + i;
      float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r[u]));
      const float2 e = *reinterpret_cast<const float2*>(tok + s);
      x = make_float2(fabsf(x.x * e.x), fabsf(x.y * e.y));
      const float2 least = make_float2(fminf(x.x, 0x1p-133f), fminf(x.y, 0x1p-133f));
      const uint32_t sign = r[u] & 0x80008000u;
#pragma unroll
      for (int v = 0; v < 3; ++v) b[ks + (u >> 1)][v][u & 1] = take_bf16(x, least) | sign;
    }
  }
}

// x / d for x < 2^31, without a division.
struct FastDiv {
  uint32_t mul, log;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t log = 0;
  while ((1ull << log) < d) ++log;
  return {(uint32_t)((((1ull << log) - d) << 32) / d + 1), log};
}
__device__ __forceinline__ int operator/(int x, FastDiv d) {
  return (int)((__umulhi((uint32_t)x, d.mul) + (uint32_t)x) >> d.log);
}

inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    return 152;
  return n;
}

}  // namespace ll
