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
#include <algorithm>
#include <type_traits>

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
  int n, N, L, out_f32;
  int split, groups, own, stages, box_rows;  // own: stages that are only the ring's
};

// A CTA serves one (row, head) for up to 8 NT nodes: eight consumer warps, and a producer warp that
// brings the pages in stages of up to 16 KB through a ring.  The products run on the tensor cores
// as out^T = page^T q^T: a page's element is brought, cut into bf16 parts and used once per node
// tile, straight from the ring, and the nodes are the narrow side.  (mma.sync, not tcgen05: the
// fp32 pages have to pass through registers to be cut, and at up to 64 nodes HBM is the bound.)
//
// Parts: q of a bf16 cache is exact, a page is two bf16 parts (to 2^-17 of each value) and so is a
// token's weight; with fp32 tokens all are three, and products down to 2^-24 are kept.  All sums are
// fp32.  Each page is summed by itself and then weighted per node, so the parts do not
// depend on the weights.
constexpr int kTreeWarps = 8, kConsumerThreads = 32 * kTreeWarps, kTreeThreads = kConsumerThreads + 32;
constexpr int kStageBytes = 16384;
constexpr int kMaxTreeStages = 8;
constexpr int kTreeSplit = 8;       // CTAs of a cluster
constexpr int kLamPitch = 32;       // levels of a node in shared memory: 7 + kMaxLevels at most

template <typename T>
struct Parts {
  static constexpr int in = sizeof(T) == 2 ? 1 : 3;      // of q, k and v
  static constexpr int page = sizeof(T) == 2 ? 2 : 3;    // of a page and of a token's weight
};

// Shared memory behind the ring's own stages, in bytes.  The tokens' weights and values are done with
// before the pages: whole stages of their place then join the ring.
struct TreeLayout {
  int kq, vp, tp;             // elements from row to row: q, v, weights
  int p, v, q, lam, pw, end;  // where each begins
};
template <typename T, int NT>
__host__ __device__ __forceinline__ TreeLayout tree_layout(int dk, int dv, int N) {
  const int dk16 = (dk + 15) & ~15, dv16 = (dv + 15) & ~15, tokens = kW + ((N + 15) & ~15);
  TreeLayout l;
  l.kq = dk16 + 8;  // an odd number of 16-byte pieces: ldmatrix without conflicts
  l.vp = dv16 + (sizeof(T) == 2 ? 8 : 4);
  l.tp = tokens + 8;
  l.p = 0;
  l.v = l.p + Parts<T>::page * 8 * NT * l.tp * 2;
  l.q = l.v + tokens * l.vp * (int)sizeof(T);
  l.lam = l.q + Parts<T>::in * 8 * NT * l.kq * 2;
  l.pw = l.lam + 8 * NT * kLamPitch * 4;
  l.end = l.pw + kMaxLevels * 8 * NT * 4;
  return l;
}

// CTAs that registers leave on an SM.
template <typename T, int NT>
constexpr int tree_ctas() { return sizeof(T) == 2 ? (NT <= 4 ? 3 : 1) : 1; }

struct TreeSmem {
  uint64_t full[kMaxTreeStages], empty[kMaxTreeStages];
  float after[kW];                   // log decay from each token of the block to the context's last
  float first[kNodes];               // log decay of the path to each node
  float la[kNodes];
  float page_log[kMaxLevels];        // the live pages, lowest level first
  int page_at[kMaxLevels], page_lv[kMaxLevels];
  int up[kNodes], depth[kNodes];
  unsigned long long above[kNodes];  // nodes on the path, itself included
  float since;
  unsigned bad[kTreeWarps + 1];      // what each warp found
  unsigned bad_tree[2];
  int odd;                           // a node's v has infinities or NaN
  int odd_q;                         // a query has
};

__device__ __forceinline__ void consumer_sync() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(kConsumerThreads) : "memory");
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3, uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix2(uint32_t& r0, uint32_t& r1, uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(at) : "memory");
}
__device__ __forceinline__ void load2(float2& v, uint32_t at) {
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
}

// x and y as bf16 parts, packed.  Cut off towards zero but for the last, and what is left of a value
// that is not 0 is never 0 or NaN (infinity less itself) but at least the least bf16: then
// infinities come out as in the sum itself.
template <int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&part)[N]) {
  const uint32_t sign = (__float_as_uint(x) >> 16 & 0x8000u) | (__float_as_uint(y) & 0x80000000u);
  float2 v = make_float2(fabsf(x), fabsf(y));
  const float2 least = make_float2(fminf(v.x, 0x1p-133f), fminf(v.y, 0x1p-133f));
#pragma unroll
  for (int i = 0; i < N - 1; ++i) part[i] = take_bf16(v, least) | sign;
  uint32_t h;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(h) : "f"(v.x), "f"(v.y));
  part[N - 1] = h | sign;
}

// The same for a page's values, in half the instructions: an infinity becomes the largest value and
// an infinity.  What is left may be 0, which only matters to an infinite query.
template <int N>
__device__ __forceinline__ void split2_page(float x, float y, uint32_t (&part)[N]) {
#pragma unroll
  for (int i = 0; i < N - 1; ++i) {
    asm("cvt.rz.satfinite.bf16x2.f32 %0, %2, %1;" : "=r"(part[i]) : "f"(x), "f"(y));
    x -= __uint_as_float(part[i] << 16);
    y -= __uint_as_float(part[i] & 0xffff0000u);
  }
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(part[N - 1]) : "f"(x), "f"(y));
}

// Fragments of mma.m16n8k16.  B from rows [n][k] in shared memory, NT tiles of 8 rows, at k0.
template <int NT>
__device__ __forceinline__ void load_b(uint32_t (&b)[NT][2], const __nv_bfloat16* rows, int pitch, int k0) {
  const int lane = threadIdx.x & 31;
  if constexpr (NT == 1) {
    ldmatrix2(b[0][0], b[0][1], tc::smem_u32(rows + (lane & 7) * pitch + k0 + ((lane >> 3) & 1) * 8));
  } else {
    const uint32_t at = tc::smem_u32(rows + ((lane & 7) + ((lane >> 4) << 3)) * pitch + k0 + ((lane >> 3) & 1) * 8);
#pragma unroll
    for (int t = 0; t < NT; t += 2) ldmatrix4(b[t][0], b[t][1], b[t + 1][0], b[t + 1][1], at + 16 * t * pitch);
  }
}
// 8 values of a row from column k on, 0 past `width`, as words of bf16 parts.
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&word)[N][4], const __nv_bfloat16* row, int k, int width, bool vec) {
  uint4 x = make_uint4(0u, 0u, 0u, 0u);
  if (vec) {
    if (k < width) x = *reinterpret_cast<const uint4*>(row + k);
  } else {
    uint32_t e[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) e[u] = k + u < width ? __bfloat16_as_ushort(row[k + u]) : 0u;
    x = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
  }
  word[0][0] = x.x;
  word[0][1] = x.y;
  word[0][2] = x.z;
  word[0][3] = x.w;
}
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&word)[N][4], const float* row, int k, int width, bool vec) {
  float e[8];
  if (vec) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    if (k < width) x = *reinterpret_cast<const float4*>(row + k);
    if (k + 4 < width) y = *reinterpret_cast<const float4*>(row + k + 4);
    e[0] = x.x; e[1] = x.y; e[2] = x.z; e[3] = x.w;
    e[4] = y.x; e[5] = y.y; e[6] = y.z; e[7] = y.w;
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u) e[u] = k + u < width ? row[k + u] : 0.f;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint32_t part[N];
    split2(e[2 * u], e[2 * u + 1], part);
#pragma unroll
    for (int j = 0; j < N; ++j) word[j][u] = part[j];
  }
}
// A from rows [k][m]: 16 tokens' values, columns m0 .. m0 + 15.
__device__ __forceinline__ void load_a_cols(uint32_t (&a)[1][4], const __nv_bfloat16* rows, int pitch, int m0) {
  const int lane = threadIdx.x & 31;
  ldmatrix_trans(a[0], rows + ((lane & 7) + ((lane >> 4) << 3)) * pitch + m0 + ((lane >> 3) & 1) * 8);
}
__device__ __forceinline__ void load_a_cols(uint32_t (&a)[3][4], const float* rows, int pitch, int m0) {
  const int lane = threadIdx.x & 31, g = lane >> 2, i = 2 * (lane & 3);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float* x = rows + (i + (u >> 1) * 8) * pitch + m0 + g + (u & 1) * 8;
    uint32_t part[3];
    split2(x[0], x[pitch], part);
#pragma unroll
    for (int j = 0; j < 3; ++j) a[j][u] = part[j];
  }
}

// The consumers' way over `rows` rows of `width` elements: f(row, first column, elements) by each
// thread in turn, 16 bytes at a time with `vec` and one element without; no divisions.
template <typename T, typename F>
__device__ __forceinline__ void over_rows(int rows, int width, bool vec, F f) {
  constexpr int per = 16 / sizeof(T);
  const int pieces = vec ? width / per : width;
  const int log = 32 - __clz(pieces - 1);  // (1 piece: 0)
  const int c = threadIdx.x & ((1 << log) - 1);
  if (c >= pieces) return;
  if (vec) {
#pragma unroll 4
    for (int r = threadIdx.x >> log; r < rows; r += kConsumerThreads >> log) f(r, c * per, per);
  } else {
#pragma unroll 4
    for (int r = threadIdx.x >> log; r < rows; r += kConsumerThreads >> log) f(r, c, 1);
  }
}
template <typename T>
__device__ __forceinline__ bool whole_pieces(const T* p, int64_t stride, int width) {
  return ((width | stride) * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}
// Rows to shared memory, asynchronously where they are whole 16-byte pieces.
template <typename T>
__device__ __forceinline__ void bring_rows(T* dst, int pitch, const T* src, int64_t stride, int rows, int width) {
  over_rows<T>(rows, width, whole_pieces(src, stride, width), [&](int r, int c, int n) {
    if (n > 1) cp_async16(dst + r * pitch + c, src + r * stride + c);
    else dst[r * pitch + c] = src[r * stride + c];
  });
}
// The queries, as bf16 parts [parts][rows][pitch], columns up to the next multiple of 16 as 0.
__device__ __forceinline__ void bring_queries(__nv_bfloat16* dst, int pitch, int /*all*/, const __nv_bfloat16* src,
                                              int64_t stride, int rows, int width) {
  bring_rows(dst, pitch, src, stride, rows, width);
  const int pad = -width & 15;
  if ((int)threadIdx.x < rows)
    for (int x = 0; x < pad; ++x) dst[threadIdx.x * pitch + width + x] = __float2bfloat16_rn(0.f);
}
__device__ __forceinline__ void bring_queries(__nv_bfloat16* dst, int pitch, int all, const float* src,
                                              int64_t stride, int rows, int width) {
  const int pairs = ((width + 15) & ~15) / 2;
  over_rows<float>(rows, pairs, false, [&](int r, int p, int) {
    const int c = 2 * p;
    uint32_t part[3];
    split2(c < width ? src[r * stride + c] : 0.f, c + 1 < width ? src[r * stride + c + 1] : 0.f, part);
#pragma unroll
    for (int j = 0; j < 3; ++j) *reinterpret_cast<uint32_t*>(dst + (j * all + r) * pitch + c) = part[j];
  });
}

// Infinity or NaN, in x or in either half of two bf16.
__device__ __forceinline__ bool is_odd(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }
__device__ __forceinline__ bool is_odd2(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}

__device__ __forceinline__ float4 load_remote4(const float* p, uint32_t rank) {
  uint32_t at;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// grid: (row, head, group of nodes, share of the cluster), the last fastest.
template <typename T, int NT>
__global__ void __launch_bounds__(kTreeThreads, tree_ctas<T, NT>())
    cache_tree_kernel(const __grid_constant__ CUtensorMap pages, ll_cache c, TreeArgs a) {
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ TreeSmem sm;
  constexpr int kIn = Parts<T>::in, kPage = Parts<T>::page, NQ = 8 * NT;
  const int H = (int)c.H, G = (int)(c.H / c.Hqk), dk = (int)c.dk, dv = (int)c.dv, M = (int)c.levels;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int Z = a.split, sp = blockIdx.x % Z, item = blockIdx.x / Z;
  const int node0 = item % a.groups * NQ, rh = item / a.groups, row = rh / H, h = rh - row * H;
  const int s = a.slots[row], pos = a.pos[row];
  if (s == -1) return;
  const unsigned why = row_bad(c, s, pos);
  const bool speaks = h == 0 && node0 == 0 && sp == 0;  // raises the row's errors
  if (why) {
    if (tid == 0 && speaks) raise(c, why);
    return;
  }
  const int N = min(a.N, node0 + NQ), queries = N - node0;  // nodes that matter here
  const int j = pos >> kLogW, r = pos & (kW - 1), par = j & 1, to = __ffs(j + 1) - 1, live = __popc(j);
  uint8_t* body = dyn + (size_t)a.own * kStageBytes;
  const TreeLayout lay = tree_layout<T, NT>(dk, dv, a.N);
  __nv_bfloat16* ps = reinterpret_cast<__nv_bfloat16*>(body + lay.p);
  T* vs = reinterpret_cast<T*>(body + lay.v);
  __nv_bfloat16* qs = reinterpret_cast<__nv_bfloat16*>(body + lay.q);
  float* lam_s = reinterpret_cast<float*>(body + lay.lam);
  float* page_w = reinterpret_cast<float*>(body + lay.pw);
  float* wt = reinterpret_cast<float*>(dyn + (size_t)(a.own - 1) * kStageBytes);  // the last own stage, until the pages need it
  float* red = reinterpret_cast<float*>(dyn);                                       // the ring, behind the pages

  // geometry of the pages: col_boxes boxes of 32 columns, the rows in stages of box_rows
  const int col_boxes = (dv + 31) / 32, box_rows = a.box_rows, box_bytes = box_rows * 128;
  const int steps = (dk + 15) / 16, share = (steps + Z - 1) / Z * 16;
  const int k0 = min(dk, sp * share), k1 = min(dk, k0 + share);  // this CTA's rows

  auto stage_at = [&](int i) { return dyn + (size_t)i * kStageBytes; };  // (those behind the ring's own: the tokens' place)
  // the producer's place in the pages: page, row; stage and how often it was used
  int m = 0, d0 = k0, st = 0, use = 0;
  auto bring_stage = [&]() {
    uint8_t* at = stage_at(st);
    tc::mbar_arrive_expect_tx(&sm.full[st], col_boxes * box_bytes);
    for (int x = 0; x < col_boxes; ++x)
      tc::tma_load_4d(&pages, &sm.full[st], at + x * box_bytes, 32 * x, d0, h, sm.page_at[m]);
    if ((d0 += box_rows) >= k1) {
      d0 = k0;
      ++m;
    }
    if (++st == a.stages) {
      st = 0;
      ++use;
    }
  };
  const T* gk = static_cast<const T*>(a.k) + row * a.sk[0] + (h / G) * a.sk[2];
  const T* gv = static_cast<const T*>(a.v) + row * a.sv[0] + h * a.sv[2];
  const T* wk = static_cast<const T*>(c.win_k) + ((int64_t)s * c.Hqk + h / G) * kW * dk;
  const T* wv = static_cast<const T*>(c.win_v) + ((int64_t)s * H + h) * kW * dv;
  const int lanes_g = lane >> 2, lanes_i = 2 * (lane & 3);
  const int tiles = kW / 16 + (N + 15) / 16;  // of 16 tokens: the block's, then the nodes; one per warp
  const bool mine = w < tiles && w % Z == sp && (w >= kW / 16 || 16 * w < r);
  const bool v_vec = whole_pieces(gv, a.sv[1], dv);
  const T* key[2];  // the thread's rows of its warp's tile: tokens g and g + 8, null where there is none
  bool key_vec = false;
  // the last two consumer warps have a node per thread: their tiles are there for most nodes only
  const int node = w < kTreeWarps ? tid - (kConsumerThreads - kNodes) : -1;
  uint32_t key_word[sizeof(T) == 2 ? 4 : 1][2][kIn][4];  // (bf16) all of them, on their way from the start
  bool ok = true;
  if (w == kTreeWarps) {
    if (lane == 0) {
      for (int i = 0; i < a.stages; ++i) {
        tc::mbar_init(&sm.full[i], 1);
        tc::mbar_init(&sm.empty[i], kTreeWarps);
      }
      tc::fence_mbar_init();
      sm.odd = 0;
      sm.odd_q = 0;
    }
    const bool here = lane < M && (j >> lane) & 1;
    const int e = here ? c.page_table[(int64_t)s * M + lane] : 0;
    const float log = here ? c.page_log[(((int64_t)s * 2 + par) * M + lane) * H + h] : 0.f;
    const bool before = before_pages(c, s, pos);
    if (here) {
      const int at = __popc(j & ((1 << lane) - 1));
      sm.page_at[at] = e;
      sm.page_lv[at] = lane;
      sm.page_log[at] = log;
    }
    const bool missing = __any_sync(0xffffffffu, e < 0 || e >= c.n_pages);
    if (lane == 0) {
      sm.bad[w] = (missing ? LL_CACHE_ERR_MISSING : 0) | (before ? LL_CACHE_ERR_POSITION : 0);
      if (!missing && k0 < k1)
        while (m < live && use == 0 && st < a.own - 1) bring_stage();
    }
    __syncwarp();
  } else {
    int up = -2;
    float la = 0.f;
    if (node >= 0 && node < a.N) {
      up = a.parents[(int64_t)row * a.N + node];
      if (a.log_a) la = a.log_a[((int64_t)row * a.N + node) * H + h];
    }
    bring_queries(qs, lay.kq, NQ, static_cast<const T*>(a.q) + row * a.sq[0] + (h / G) * a.sq[2] + node0 * a.sq[1],
                  a.sq[1], queries, dk);
    for (int q = w; q < queries; q += kTreeWarps)
      if (lane < M + kLogW + 1)
        tc::cp_async4(lam_s + q * kLamPitch + lane, a.lam + (((int64_t)row * a.N + node0 + q) * H + h) * a.L + lane, 4);
    cp_async_commit();
    bring_rows(vs, lay.vp, wv, dv, r, dv);
    bring_rows(vs + kW * lay.vp, lay.vp, gv, a.sv[1], N, dv);
    cp_async_commit();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = 16 * w + lanes_g + 8 * u;
      key[u] = !mine ? nullptr : x < kW ? (x < r ? wk + x * dk : nullptr) : x - kW < N ? gk + (x - kW) * a.sk[1] : nullptr;
    }
    key_vec = w < kW / 16 ? whole_pieces(wk, dk, dk) : whole_pieces(gk, a.sk[1], dk);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int u = 0; u < 2; ++u) load_words(key_word[d][u], key[u], 32 * d + 4 * lanes_i, key[u] ? dk : 0, key_vec);
    }
    // no tokens, no values: up to a whole tile behind the block's and the nodes
    over_rows<T>(-r & 15, dv, false, [&](int y, int x, int) { vs[(r + y) * lay.vp + x] = from_f32<T>(0.f); });
    over_rows<T>(-N & 15, dv, false, [&](int y, int x, int) { vs[(kW + N + y) * lay.vp + x] = from_f32<T>(0.f); });
    unsigned bad = 0;
    if (node >= 0) {
      const bool fine = up < node && up >= -2;
      if (!fine) bad = LL_CACHE_ERR_TREE;
      sm.up[node] = fine ? up : -2;
      sm.la[node] = up != -2 ? la : 0.f;
    } else if (w == 0) {
      float since;
      block_decays(c.win_log_a + ((int64_t)s * H + h) * kW, r, c.page_from[s * 2 + par], sm.after, &since);
      if (lane == 0) sm.since = since;
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (lane == 0) sm.bad[w] = bad;
    cp_async_wait<1>();
  }
  __syncthreads();
  if (node >= 0) {  // the nodes' paths; weights and log decays along those of the queries
    unsigned long long above = 0;
    unsigned bad = 0;
    int depth = -1;
    const bool in = sm.up[node] != -2;
    for (int x = node; in && x >= 0; x = sm.up[x]) {
      above |= 1ull << x;
      ++depth;
      if (sm.up[x] == -2) bad = LL_CACHE_ERR_TREE;  // a child of a node that is left out
    }
    const int q = node - node0, t = pos + depth;
    if (in && !position_ok(c, t)) bad |= LL_CACHE_ERR_POSITION;
    sm.above[node] = above;
    sm.depth[node] = depth;
    if (in && !bad && q >= 0 && q < queries) {
      float acc = 0.f;  // log a behind x up to the node
      for (int x = node, tx = t; x >= 0; x = sm.up[x], --tx) {
        wt[q * kNodes + x] = lam_s[q * kLamPitch + fenwick_level(t, tx)] * expf(acc);
        acc += sm.la[x];
      }
      sm.first[node] = acc;
    }
    tc::fence_proxy_async_smem();  // the stage's pages are written behind the weights
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (lane == 0) sm.bad_tree[w - (kTreeWarps - 2)] = bad;
  } else if (w < kTreeWarps) {  // queries that are infinite or NaN
    bool odd = false;
    for (int q = w; q < queries; q += kTreeWarps - 2)
      for (int x = 2 * lane; x < dk; x += 64)
#pragma unroll
        for (int y = 0; y < kIn; ++y) odd |= is_odd2(*reinterpret_cast<const uint32_t*>(qs + (y * NQ + q) * lay.kq + x));
    if (odd) sm.odd_q = 1;
  }
  float sc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int u = 0; u < 4; ++u) sc[t][u] = 0.f;
  // scores of 16 tokens per warp, K q^T, not yet weighted.  Each thread has 8 neighbouring values of a row, so the
  // sum goes over them in another order than the fragments': the same for keys and queries.
  if (mine) {
    const int dk16 = (dk + 15) & ~15;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const int at = 32 * d + 4 * lanes_i;
      if (32 * d >= dk) break;
      uint32_t kw[2][kIn][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int x = 0; x < 4; ++x) kw[u][0][x] = key_word[d][u][0][x];
        } else {
          load_words(kw[u], key[u], at, key[u] ? dk : 0, key_vec);
        }
      }
#pragma unroll
      for (int y = kIn - 1; y >= 0; --y)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint4 q = make_uint4(0u, 0u, 0u, 0u);
          if (at < dk16) q = *reinterpret_cast<const uint4*>(qs + (y * NQ + 8 * t + lanes_g) * lay.kq + at);
#pragma unroll
          for (int x = kIn - 1 - y; x >= 0; --x) {
            const uint32_t lo[4] = {kw[0][x][0], kw[1][x][0], kw[0][x][1], kw[1][x][1]};
            const uint32_t hi[4] = {kw[0][x][2], kw[1][x][2], kw[0][x][3], kw[1][x][3]};
            mma_bf16(sc[t], lo, q.x, q.y);
            mma_bf16(sc[t], hi, q.z, q.w);
          }
        }
    }
  }
  __syncthreads();
  unsigned bad = sm.bad_tree[0] | sm.bad_tree[1];
#pragma unroll
  for (int i = 0; i <= kTreeWarps; ++i) bad |= sm.bad[i];
  if (bad) {
    if (tid == 0 && speaks) raise(c, bad);
    if (w == kTreeWarps) {
      for (int i = 0; lane == 0 && i < st; ++i) tc::mbar_wait_short(&sm.full[i], 0);  // the copies on their way
    } else {
      cp_async_wait<0>();
    }
    return;
  }

  if (w == kTreeWarps) {
    if (lane == 0 && k0 < k1) {
      while (m < live) {
        // the last own stage and those behind it have one more release, of what they hold first
        const int released = use + (st >= a.own - 1);
        if (released && !(ok = tc::mbar_wait_short(&sm.empty[st], (released - 1) & 1))) break;
        bring_stage();
      }
      if (!ok) {
        raise(c, LL_CACHE_ERR_WAIT);
        for (int i = 0; i < a.stages; ++i) {  // the copies on their way end before the CTA does
          const int uses = use + (i < st);
          if (uses) tc::mbar_wait_short(&sm.full[i], (uses - 1) & 1);
        }
      }
    }
    __syncwarp();
  } else {
    // the weighted scores
    if (mine) {
      const bool nodes = w >= kW / 16;
      const int x0 = 16 * w + lanes_g - (nodes ? kW : 0);  // the thread's tokens: x0 and x0 + 8
      const float after0 = nodes ? 0.f : sm.after[x0], after1 = nodes ? 0.f : sm.after[x0 + 8];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int q = 8 * t + lanes_i;
        float2 f[2];  // [token][node]
        if (nodes) {
          const unsigned long long a0 = sm.above[node0 + q] >> x0, a1 = sm.above[node0 + q + 1] >> x0;
          f[0].x = a0 & 1 ? wt[q * kNodes + x0] * sc[t][0] : 0.f;
          f[0].y = a1 & 1 ? wt[(q + 1) * kNodes + x0] * sc[t][1] : 0.f;
          f[1].x = a0 >> 8 & 1 ? wt[q * kNodes + x0 + 8] * sc[t][2] : 0.f;
          f[1].y = a1 >> 8 & 1 ? wt[(q + 1) * kNodes + x0 + 8] * sc[t][3] : 0.f;
        } else {
          const int2 depth = *reinterpret_cast<const int2*>(&sm.depth[node0 + q]);
          const float2 first = *reinterpret_cast<const float2*>(&sm.first[node0 + q]);
          const float* lam0 = lam_s + q * kLamPitch;
          const int t0 = pos + depth.x, t1 = pos + depth.y, s0 = (j << kLogW) + x0, s1 = s0 + 8;
          f[0].x = depth.x >= 0 && s0 < pos ? lam0[fenwick_level(t0, s0)] * expf(after0 + first.x) * sc[t][0] : 0.f;
          f[1].x = depth.x >= 0 && s1 < pos ? lam0[fenwick_level(t0, s1)] * expf(after1 + first.x) * sc[t][2] : 0.f;
          lam0 += kLamPitch;
          f[0].y = depth.y >= 0 && s0 < pos ? lam0[fenwick_level(t1, s0)] * expf(after0 + first.y) * sc[t][1] : 0.f;
          f[1].y = depth.y >= 0 && s1 < pos ? lam0[fenwick_level(t1, s1)] * expf(after1 + first.y) * sc[t][3] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t part[kPage];
          split2(f[u].x, f[u].y, part);
          __nv_bfloat16* at = ps + q * lay.tp + 16 * w + lanes_g + 8 * u;
#pragma unroll
          for (int x = 0; x < kPage; ++x) {
            at[x * NQ * lay.tp] = __ushort_as_bfloat16((unsigned short)(part[x] & 0xffffu));
            at[x * NQ * lay.tp + lay.tp] = __ushort_as_bfloat16((unsigned short)(part[x] >> 16));
          }
        }
      }
    }
    for (int x = tid; x < live * NQ; x += kConsumerThreads) {
      const int y = x / NQ, q = x - y * NQ, i = node0 + q;
      float f = 0.f;
      if (q < queries && sm.up[i] != -2) {
        const int lv = (pos + sm.depth[i]) >> kLogW > j ? max(sm.page_lv[y], to) : sm.page_lv[y];
        f = lam_s[q * kLamPitch + kLogW + 1 + lv] * expf(sm.page_log[y] + sm.since + sm.first[i]);
      }
      page_w[x] = f;
    }
    // values of nodes, each thread the ones it brought: none where a node is left out; infinities and
    // NaN go by themselves, to the nodes below them alone
    cp_async_wait<0>();
    over_rows<T>(N, dv, v_vec, [&](int y, int x, int n) {
      T* p = vs + (kW + y) * lay.vp + x;
      const bool out = sm.up[y] == -2;
      if (n > 1) {
        uint4 v = *reinterpret_cast<const uint4*>(p);
        bool odd;
        if constexpr (sizeof(T) == 2) odd = is_odd2(v.x) || is_odd2(v.y) || is_odd2(v.z) || is_odd2(v.w);
        else odd = is_odd(__uint_as_float(v.x)) || is_odd(__uint_as_float(v.y)) || is_odd(__uint_as_float(v.z)) || is_odd(__uint_as_float(v.w));
        if (odd || out) {
          if (!out) sm.odd = 1;
#pragma unroll
          for (int u = 0; u < 16 / (int)sizeof(T); ++u)
            if (out || is_odd(to_f32(p[u]))) p[u] = from_f32<T>(0.f);
        }
      } else if (out || is_odd(to_f32(*p))) {
        if (!out) sm.odd = 1;
        *p = from_f32<T>(0.f);
      }
    });
    consumer_sync();  // the tokens' weights and values are there, the tree's weights are done with
    if (lane == 0) tc::mbar_arrive(&sm.empty[a.own - 1]);

    // a warp's 16 columns; where there are few, warps share them by tokens and by rows of the pages
    const int cols = (dv + 15) / 16, wide = cols > 4 ? 8 : cols > 2 ? 4 : cols;
    const int ct = w & (wide - 1), kp = w / wide, kparts = kTreeWarps / wide;
    const bool on = ct < cols;
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int u = 0; u < 4; ++u) acc[t][u] = 0.f;
    if (on) {
      int turn = 0;
      for (int tile = sp; tile < tiles; tile += Z) {
        if (tile < kW / 16 && 16 * tile >= r) continue;
        if (turn++ % kparts != kp) continue;
        uint32_t va[kIn][4];
        load_a_cols(va, vs + 16 * tile * lay.vp, lay.vp, 16 * ct);
#pragma unroll
        for (int y = kPage - 1; y >= 0; --y) {
          uint32_t pb[NT][2];
          load_b<NT>(pb, ps + y * NQ * lay.tp, lay.tp, 16 * tile);
#pragma unroll
          for (int x = kIn - 1; x >= 0; --x)
            if (x + y < kPage)
#pragma unroll
              for (int t = 0; t < NT; ++t) mma_bf16(acc[t], va[x], pb[t][0], pb[t][1]);
        }
      }
    }
    // from columns g and g + 8 of each thread to 2 g and 2 g + 1, as the pages come
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int src = (((2 * lanes_g + (u >> 1)) & 7) << 2) | (lane & 3);
        const float lo = __shfl_sync(0xffffffffu, acc[t][u & 1], src), hi = __shfl_sync(0xffffffffu, acc[t][2 + (u & 1)], src);
        y[u] = lanes_g < 4 ? lo : hi;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) acc[t][u] = y[u];
    }
    const int col = 16 * ct + 2 * lanes_g;
    if (sm.odd && on && kp == 0 && col < dv) {
      for (int y = 0; y < N; ++y) {
        if ((kW + y) / 16 % Z != sp) continue;
        const float v0 = to_f32(gv[y * a.sv[1] + col]), v1 = to_f32(gv[y * a.sv[1] + col + 1]);
        if (!is_odd(v0) && !is_odd(v1)) continue;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int q = 8 * t + lanes_i + (u & 1);
            const float v = u >> 1 ? v1 : v0;
            if (q >= queries || !(sm.above[node0 + q] >> y & 1) || !is_odd(v)) continue;
            float p = 0.f;
            for (int x = kPage - 1; x >= 0; --x) p += to_f32(ps[(x * NQ + q) * lay.tp + kW + y]);
            acc[t][u] = fmaf(p, v, acc[t][u]);
          }
      }
    }

    if (a.stages > a.own) {  // the tokens' weights and values are done with
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0)
        for (int i = a.own; i < a.stages; ++i) tc::mbar_arrive(&sm.empty[i]);
    }

    // the pages.  A warp takes two neighbouring steps of 16 rows of each stage (one where eight warps share
    // a column tile); addresses are kept as shared-memory offsets, in steps of a stage.
    const int chunk = 4 * (ct & 1) + (lanes_g >> 1);
    const uint32_t rows_at = tc::smem_u32(dyn) + (ct >> 1) * box_bytes + (lanes_g & 1) * 8 + 2048 * (wide > 1 ? 2 * kp : kp);
    const uint32_t off0 = tc::sw128_offset(lanes_i, chunk), off1 = tc::sw128_offset(lanes_i + 1, chunk);
    const int first_row = 16 * (wide > 1 ? 2 * kp : kp);
    const uint32_t q_at = tc::smem_u32(qs) + ((lane & 7) + (NT > 1 ? (lane >> 4) << 3 : 0)) * lay.kq * 2 +
                          ((lane >> 3) & 1) * 16 + 2 * first_row;
    const uint32_t q_tiles = 16 * lay.kq * 2, q_parts = NQ * lay.kq * 2;
    auto over_pages = [&](auto robust) {
      int stage = 0, phase = 0;
      for (int x = 0; x < live; ++x) {
        float part[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int u = 0; u < 4; ++u) part[t][u] = 0.f;
        for (int d = k0; d < k1; d += box_rows) {
          if (ok) ok = tc::mbar_wait_short(&sm.full[stage], phase);
          const uint32_t at = rows_at + stage * kStageBytes, qa = q_at + 2 * d;
          const int rows = min(box_rows, k1 - d) - first_row;  // from this warp's first on
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            if (!on || 16 * z >= rows || (z && wide == 1)) continue;
            float2 v[4];
            load2(v[0], at + off0 + 2048 * z);
            load2(v[1], at + off1 + 2048 * z);
            load2(v[2], at + off0 + 2048 * z + 1024);
            load2(v[3], at + off1 + 2048 * z + 1024);
            uint32_t pa[kPage][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t cut[kPage];
              const float lo = u & 1 ? v[u & 2].y : v[u & 2].x, hi = u & 1 ? v[(u & 2) + 1].y : v[(u & 2) + 1].x;
              if constexpr (decltype(robust)::value) split2(lo, hi, cut);
              else split2_page(lo, hi, cut);
#pragma unroll
              for (int y = 0; y < kPage; ++y) pa[y][u] = cut[y];
            }
#pragma unroll
            for (int y = kIn - 1; y >= 0; --y) {
              uint32_t qb[NT][2];
              const uint32_t q = qa + y * q_parts + 32 * z;
              if constexpr (NT == 1) {
                ldmatrix2(qb[0][0], qb[0][1], q);
              } else {
#pragma unroll
                for (int t = 0; t < NT; t += 2) ldmatrix4(qb[t][0], qb[t][1], qb[t + 1][0], qb[t + 1][1], q + (t / 2) * q_tiles);
              }
#pragma unroll
              for (int u = kPage - 1; u >= 0; --u)
                if (u + y < kPage)
#pragma unroll
                  for (int t = 0; t < NT; ++t) mma_bf16(part[t], pa[u], qb[t][0], qb[t][1]);
            }
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.empty[stage]);
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float2 f = *reinterpret_cast<const float2*>(page_w + x * NQ + 8 * t + lanes_i);
          acc[t][0] = fmaf(f.x, part[t][0], acc[t][0]);
          acc[t][1] = fmaf(f.y, part[t][1], acc[t][1]);
          acc[t][2] = fmaf(f.x, part[t][2], acc[t][2]);
          acc[t][3] = fmaf(f.y, part[t][3], acc[t][3]);
        }
      }
    };
    if (k0 < k1) {
      if (sm.odd_q) over_pages(std::true_type());
      else over_pages(std::false_type());
    }
    if (!ok && lane == 0) raise(c, LL_CACHE_ERR_WAIT);

    // sums over the warps that share columns, and over the cluster
    const bool pairs = (reinterpret_cast<uintptr_t>(a.out) & (a.out_f32 ? 7u : 3u)) == 0;
    auto put = [&](int t, int ct_, const float (&x)[4]) {
      const int col_ = 16 * ct_ + 2 * lanes_g;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int q = 8 * t + lanes_i + u;
        if (q >= queries || col_ >= dv || sm.up[node0 + q] == -2) continue;
        const int64_t at = (((int64_t)row * a.N + node0 + q) * H + h) * dv + col_;
        if (a.out_f32) {
          float* o = static_cast<float*>(a.out) + at;
          if (pairs) {
            *reinterpret_cast<float2*>(o) = make_float2(x[u], x[2 + u]);
          } else {
            o[0] = x[u];
            o[1] = x[2 + u];
          }
        } else {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + at;
          if (pairs) {
            *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(x[u], x[2 + u]);
          } else {
            o[0] = __float2bfloat16_rn(x[u]);
            o[1] = __float2bfloat16_rn(x[2 + u]);
          }
        }
      }
    };
    if (kparts == 1 && Z == 1) {
      if (on)
#pragma unroll
        for (int t = 0; t < NT; ++t) put(t, ct, acc[t]);
    } else {
      consumer_sync();  // the ring is done with
#pragma unroll
      for (int t = 0; t < NT; ++t)
        *reinterpret_cast<float4*>(red + ((t * kTreeWarps + w) * 32 + lane) * 4) = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
      if (Z == 1) {
        consumer_sync();
        for (int x = w; x < NT * cols; x += kTreeWarps) {
          const int t = x / cols, ct_ = x - t * cols;
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int p = 0; p < kparts; ++p)
            y = add4(y, *reinterpret_cast<const float4*>(red + ((t * kTreeWarps + p * wide + ct_) * 32 + lane) * 4));
          const float z[4] = {y.x, y.y, y.z, y.w};
          put(t, ct_, z);
        }
      }
    }
    if (Z > 1) {
      __syncwarp();
      cluster_arrive();
      cluster_wait();
      for (int x = w * Z + sp; x < NT * cols; x += kTreeWarps * Z) {
        const int t = x / cols, ct_ = x - t * cols;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int z = 0; z < Z; ++z)
          for (int p = 0; p < kparts; ++p)
            y = add4(y, load_remote4(red + ((t * kTreeWarps + p * wide + ct_) * 32 + lane) * 4, z));
        const float z[4] = {y.x, y.y, y.z, y.w};
        put(t, ct_, z);
      }
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    }
  }
  if (w == kTreeWarps && Z > 1) {
    cluster_arrive();
    cluster_wait();
    cluster_arrive();
    cluster_wait();
  }
}

// CTAs per item: doubled while that leaves the launch within the SMs, each with at least 16 rows of the pages.
int tree_split(int64_t items, int dk, int sms) {
  int split = 1;
  while (split < kTreeSplit && items * split * 2 <= sms && dk > 16 * split) split *= 2;
  return split;
}

constexpr size_t kSm = 233472;  // shared memory of an SM

template <typename T, int NT>
cudaError_t launch(const ll_cache& c, TreeArgs a, cudaStream_t s) {
  const int dk = (int)c.dk, dv = (int)c.dv;
  a.groups = (a.N + 8 * NT - 1) / (8 * NT);
  const int64_t items = (int64_t)a.n * c.H * a.groups;
  a.split = tree_split(items, dk, sm_count());
  const int share = ((dk + 15) / 16 + a.split - 1) / a.split * 16;
  const int col_boxes = (dv + 31) / 32;
  a.box_rows = std::min(col_boxes == 1 ? 128 : col_boxes == 2 ? 64 : 32, share);  // a stage, or a CTA's share
  const TreeLayout lay = tree_layout<T, NT>(dk, dv, a.N);
  const size_t fixed = sizeof(TreeSmem) + 2048;  // (1024 of each CTA are the system's)
  // as many CTAs on an SM as leave the ring three stages, one of them from the start
  const int later = lay.q / kStageBytes;
  int ctas = tree_ctas<T, NT>();
  while (ctas > 1 && fixed + lay.end + std::max(1, 3 - later) * kStageBytes > kSm / ctas) --ctas;
  a.own = (int)std::min<size_t>(kMaxTreeStages, (kSm / ctas - fixed - lay.end) / kStageBytes);
  a.stages = std::min(kMaxTreeStages, a.own + later);
  const size_t smem = (size_t)a.own * kStageBytes + lay.end;
  CUtensorMap pages;
  if (!make_pages_map(&pages, c.pages, c.n_pages, c.H, c.dk, c.dv, a.box_rows)) return cudaErrorInvalidValue;
  const auto kernel = cache_tree_kernel<T, NT>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_following(false, kernel, dim3((unsigned)(items * a.split)), kTreeThreads, smem, a.split, s, pages, c, a);
}

}  // namespace

cudaError_t launch_cache_tree(const ll_cache& c, const int* slots, const int* pos, const int* parents,
                              const void* q, const int64_t* sq, const void* k, const int64_t* sk,
                              const void* v, const int64_t* sv, const float* log_a, const float* lam,
                              void* out, int n, int N, int L, int out_dtype, cudaStream_t s) {
  TreeArgs a = {};
  a.slots = slots; a.pos = pos; a.parents = parents; a.q = q; a.k = k; a.v = v; a.log_a = log_a;
  a.lam = lam; a.out = out; a.n = n; a.N = N; a.L = L; a.out_f32 = out_dtype == LL_F32;
  for (int i = 0; i < 3; ++i) {
    a.sq[i] = sq[i];
    a.sk[i] = sk[i];
    a.sv[i] = sv[i];
  }
  if (c.dtype == LL_F32)  // (three parts of everything: 32 nodes are what shared memory and registers hold)
    return N <= 8 ? launch<float, 1>(c, a, s) : N <= 16 ? launch<float, 2>(c, a, s) : launch<float, 4>(c, a, s);
  return N <= 8 ? launch<__nv_bfloat16, 1>(c, a, s) : N <= 16 ? launch<__nv_bfloat16, 2>(c, a, s)
         : N <= 32 ? launch<__nv_bfloat16, 4>(c, a, s) : launch<__nv_bfloat16, 8>(c, a, s);
}

}  // namespace ll
