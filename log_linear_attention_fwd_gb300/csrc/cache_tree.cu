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
  int split, groups, stages, box_log;
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

// Shared memory behind the ring, in bytes.
struct TreeLayout {
  int kq, vp, tp;                // elements from row to row: q and k, v, weights
  int q, k, v, lam, pw, end;     // where each begins; the weights' parts and the last sums take k's place
};
template <typename T, int NT>
__host__ __device__ __forceinline__ TreeLayout tree_layout(int dk, int dv, int N) {
  const int dk16 = (dk + 15) & ~15, dv16 = (dv + 15) & ~15, tokens = kW + ((N + 15) & ~15);
  TreeLayout l;
  l.kq = dk16 + 8;  // an odd number of 16-byte pieces: ldmatrix without conflicts
  l.vp = dv16 + (sizeof(T) == 2 ? 8 : 4);
  l.tp = tokens + 8;
  l.q = 0;
  l.k = l.q + Parts<T>::in * 8 * NT * l.kq * 2;
  int k = tokens * l.kq * (int)sizeof(T);
  const int p = Parts<T>::page * 8 * NT * l.tp * 2, red = kTreeWarps * NT * 512;
  k = k > p ? k : p;
  l.v = l.k + (k > red ? k : red);
  l.lam = l.v + tokens * l.vp * (int)sizeof(T);
  l.pw = l.lam + 8 * NT * kLamPitch * 4;
  l.end = l.pw + kMaxLevels * 8 * NT * 4;
  return l;
}

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
  unsigned bad;
  int odd;                           // a node's v has infinities or NaN
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
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const __nv_bfloat16* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(tc::smem_u32(p))
               : "memory");
}
__device__ __forceinline__ void ldmatrix2(uint32_t& r0, uint32_t& r1, const __nv_bfloat16* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];"
               : "=r"(r0), "=r"(r1)
               : "r"(tc::smem_u32(p))
               : "memory");
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

// Fragments of mma.m16n8k16.  B from rows [n][k] in shared memory, NT tiles of 8 rows, at k0.
template <int NT>
__device__ __forceinline__ void load_b(uint32_t (&b)[NT][2], const __nv_bfloat16* rows, int pitch, int k0) {
  const int lane = threadIdx.x & 31;
  if constexpr (NT == 1) {
    ldmatrix2(b[0][0], b[0][1], rows + (lane & 7) * pitch + k0 + ((lane >> 3) & 1) * 8);
  } else {
#pragma unroll
    for (int t = 0; t < NT; t += 2) {
      uint32_t r[4];
      ldmatrix4(r, rows + (8 * t + (lane & 7) + ((lane >> 4) << 3)) * pitch + k0 + ((lane >> 3) & 1) * 8);
      b[t][0] = r[0];
      b[t][1] = r[1];
      b[t + 1][0] = r[2];
      b[t + 1][1] = r[3];
    }
  }
}
// A from rows [m][k]: 16 tokens' keys.
__device__ __forceinline__ void load_a_rows(uint32_t (&a)[1][4], const __nv_bfloat16* rows, int pitch, int k0) {
  const int lane = threadIdx.x & 31;
  ldmatrix4(a[0], rows + ((lane & 7) + ((lane >> 3) & 1) * 8) * pitch + k0 + (lane >> 4) * 8);
}
__device__ __forceinline__ void load_a_rows(uint32_t (&a)[3][4], const float* rows, int pitch, int k0) {
  const int lane = threadIdx.x & 31, g = lane >> 2, i = 2 * (lane & 3);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float2 x = *reinterpret_cast<const float2*>(rows + (g + (u & 1) * 8) * pitch + k0 + i + (u >> 1) * 8);
    uint32_t part[3];
    split2(x.x, x.y, part);
#pragma unroll
    for (int j = 0; j < 3; ++j) a[j][u] = part[j];
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

// `rows` rows of `width` elements to shared memory, by the consumers: asynchronously where all are
// whole 16-byte pieces; columns up to the next multiple of 16 become 0 with zero_pad.
template <typename T>
__device__ __forceinline__ void bring_rows(T* dst, int pitch, const T* src, int64_t stride, int rows, int width,
                                           bool zero_pad) {
  constexpr int per = 16 / sizeof(T);
  if (width % per == 0 && (stride * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
    const int chunks = width / per;
    for (int x = threadIdx.x; x < rows * chunks; x += kConsumerThreads) {
      const int r = x / chunks, c = (x - r * chunks) * per;
      cp_async16(dst + r * pitch + c, src + r * stride + c);
    }
  } else {
#pragma unroll 4
    for (int x = threadIdx.x; x < rows * width; x += kConsumerThreads) {
      const int r = x / width;
      dst[r * pitch + x - r * width] = src[r * stride + (x - r * width)];
    }
  }
  const int pad = zero_pad ? (16 - (width & 15)) & 15 : 0;
  for (int x = threadIdx.x; x < rows * pad; x += kConsumerThreads)
    dst[x / pad * pitch + width + x % pad] = from_f32<T>(0.f);
}
// The queries, as bf16 parts [parts][rows][pitch].
__device__ __forceinline__ void bring_queries(__nv_bfloat16* dst, int pitch, int /*all*/, const __nv_bfloat16* src,
                                              int64_t stride, int rows, int width) {
  bring_rows(dst, pitch, src, stride, rows, width, true);
}
__device__ __forceinline__ void bring_queries(__nv_bfloat16* dst, int pitch, int all, const float* src,
                                              int64_t stride, int rows, int width) {
  const int pairs = ((width + 15) & ~15) / 2;
#pragma unroll 4
  for (int x = threadIdx.x; x < rows * pairs; x += kConsumerThreads) {
    const int r = x / pairs, c = 2 * (x - r * pairs);
    uint32_t part[3];
    split2(c < width ? src[r * stride + c] : 0.f, c + 1 < width ? src[r * stride + c + 1] : 0.f, part);
#pragma unroll
    for (int j = 0; j < 3; ++j) *reinterpret_cast<uint32_t*>(dst + (j * all + r) * pitch + c) = part[j];
  }
}

__device__ __forceinline__ bool is_odd(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

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
__global__ void __launch_bounds__(kTreeThreads, sizeof(T) == 2 && NT <= 4 ? 2 : 1)
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
  uint8_t* body = dyn + (size_t)a.stages * kStageBytes;
  const TreeLayout lay = tree_layout<T, NT>(dk, dv, a.N);
  __nv_bfloat16* qs = reinterpret_cast<__nv_bfloat16*>(body + lay.q);
  T* ks = reinterpret_cast<T*>(body + lay.k);
  __nv_bfloat16* ps = reinterpret_cast<__nv_bfloat16*>(body + lay.k);
  float* red = reinterpret_cast<float*>(body + lay.k);
  T* vs = reinterpret_cast<T*>(body + lay.v);
  float* lam_s = reinterpret_cast<float*>(body + lay.lam);
  float* page_w = reinterpret_cast<float*>(body + lay.pw);
  float* wt = reinterpret_cast<float*>(dyn + (size_t)(a.stages - 1) * kStageBytes);  // the last stage, until the pages need it

  // geometry of the pages: col_boxes boxes of 32 columns, the rows in stages of `span`
  const int col_boxes = (dv + 31) / 32, box_log = a.box_log, box_rows = 1 << box_log, box_bytes = box_rows * 128;
  const int span = col_boxes == 1 ? 128 : col_boxes == 2 ? 64 : 32;
  const int steps = (dk + 15) / 16, share = (steps + Z - 1) / Z * 16;
  const int k0 = min(dk, sp * share), k1 = min(dk, k0 + share);  // this CTA's rows

  if (tid == 0) {
    for (int i = 0; i < a.stages; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.empty[i], kTreeWarps);
    }
    tc::fence_mbar_init();
    sm.bad = before_pages(c, s, pos) ? LL_CACHE_ERR_POSITION : 0;
    sm.odd = 0;
  }
  __syncthreads();

  // the producer's place in the pages: page, row; stage and how often it was used
  int m = 0, d0 = k0, st = 0, use = 0;
  auto bring_stage = [&]() {
    const int rows = min(span, k1 - d0), boxes = (rows + box_rows - 1) >> box_log;
    uint8_t* to_ = dyn + (size_t)st * kStageBytes;
    tc::mbar_arrive_expect_tx(&sm.full[st], boxes * col_boxes * box_bytes);
    for (int b = 0; b < boxes; ++b)
      for (int x = 0; x < col_boxes; ++x)
        tc::tma_load_4d(&pages, &sm.full[st], to_ + (b * col_boxes + x) * box_bytes, 32 * x, d0 + b * box_rows, h,
                        sm.page_at[m]);
    if ((d0 += span) >= k1) {
      d0 = k0;
      ++m;
    }
    if (++st == a.stages) {
      st = 0;
      ++use;
    }
  };
  bool ok = true;
  if (w == kTreeWarps) {
    const bool here = lane < M && (j >> lane) & 1;
    const int e = here ? c.page_table[(int64_t)s * M + lane] : 0;
    const float log = here ? c.page_log[(((int64_t)s * 2 + par) * M + lane) * H + h] : 0.f;
    if (here) {
      const int at = __popc(j & ((1 << lane) - 1));
      sm.page_at[at] = e;
      sm.page_lv[at] = lane;
      sm.page_log[at] = log;
    }
    const bool missing = __any_sync(0xffffffffu, e < 0 || e >= c.n_pages);
    if (missing && lane == 0) atomicOr(&sm.bad, LL_CACHE_ERR_MISSING);
    if (!missing && lane == 0 && k0 < k1)
      while (m < live && use == 0 && st < a.stages - 1) bring_stage();
    __syncwarp();
  } else {
    const T* gq = static_cast<const T*>(a.q) + row * a.sq[0] + (h / G) * a.sq[2] + node0 * a.sq[1];
    const T* gk = static_cast<const T*>(a.k) + row * a.sk[0] + (h / G) * a.sk[2];
    const T* gv = static_cast<const T*>(a.v) + row * a.sv[0] + h * a.sv[2];
    const T* wk = static_cast<const T*>(c.win_k) + ((int64_t)s * c.Hqk + h / G) * kW * dk;
    const T* wv = static_cast<const T*>(c.win_v) + ((int64_t)s * H + h) * kW * dv;
    bring_queries(qs, lay.kq, NQ, gq, a.sq[1], queries, dk);
    bring_rows(ks, lay.kq, wk, dk, r, dk, true);
    bring_rows(ks + kW * lay.kq, lay.kq, gk, a.sk[1], N, dk, true);
    cp_async_commit();
    bring_rows(vs, lay.vp, wv, dv, r, dv, false);
    bring_rows(vs + kW * lay.vp, lay.vp, gv, a.sv[1], N, dv, false);
    cp_async_commit();
    for (int x = tid; x < (((r + 15) & ~15) - r) * dv; x += kConsumerThreads)  // no tokens: no values
      vs[(r + x / dv) * lay.vp + x % dv] = from_f32<T>(0.f);
    if (tid < kNodes) {
      const int up = tid < a.N ? a.parents[(int64_t)row * a.N + tid] : -2;
      const bool fine = up < tid && up >= -2;
      if (!fine) atomicOr(&sm.bad, LL_CACHE_ERR_TREE);
      sm.up[tid] = fine ? up : -2;
      sm.la[tid] = fine && up != -2 && a.log_a ? a.log_a[((int64_t)row * a.N + tid) * H + h] : 0.f;
    } else if (w == 2) {
      float since;
      block_decays(c.win_log_a + ((int64_t)s * H + h) * kW, r, c.page_from[s * 2 + par], sm.after, &since);
      if (lane == 0) sm.since = since;
    }
    for (int x = tid; x < queries * kLamPitch; x += kConsumerThreads)
      if (x % kLamPitch < M + kLogW + 1)
        lam_s[x] = a.lam[(((int64_t)row * a.N + node0 + x / kLamPitch) * H + h) * a.L + x % kLamPitch];
  }
  __syncthreads();
  if (tid < kNodes) {
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
    if (tid == 0 && speaks) raise(c, sm.bad);
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
        // the last stage has one more release: of the tree's weights
        const int released = use + (st == a.stages - 1);
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
    // log decays of the paths, and the weight of every node above another: sums along the path
    if (tid < queries && sm.up[node0 + tid] != -2) {
      const int i = node0 + tid, t = pos + sm.depth[i];
      float acc = 0.f;  // log a behind x up to the node
      for (int x = i; x >= 0; x = sm.up[x]) {
        wt[tid * kNodes + x] = lam_s[tid * kLamPitch + fenwick_level(t, pos + sm.depth[x])] * expf(acc);
        acc += sm.la[x];
      }
      sm.first[i] = acc;
      tc::fence_proxy_async_smem();  // the stage's pages are written behind the weights
    }
    cp_async_wait<1>();
    consumer_sync();
    // scores of 16 tokens per warp, K q^T, weighted
    const int lanes_g = lane >> 2, lanes_i = 2 * (lane & 3);
    const int tiles = kW / 16 + (N + 15) / 16;  // of tokens: the block's, then the nodes
    const bool mine = w < tiles && w % Z == sp && (w >= kW / 16 || 16 * w < r);
    float sc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int u = 0; u < 4; ++u) sc[t][u] = 0.f;
    if (mine) {
      for (int d = 0; d < dk; d += 16) {
        uint32_t ka[kIn][4];
        load_a_rows(ka, ks + 16 * w * lay.kq, lay.kq, d);
#pragma unroll
        for (int y = kIn - 1; y >= 0; --y) {
          uint32_t qb[NT][2];
          load_b<NT>(qb, qs + y * NQ * lay.kq, lay.kq, d);
#pragma unroll
          for (int x = kIn - 1 - y; x >= 0; --x)
#pragma unroll
            for (int t = 0; t < NT; ++t) mma_bf16(sc[t], ka[x], qb[t][0], qb[t][1]);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int q = 8 * t + lanes_i + (u & 1), x = 16 * w + lanes_g + (u >> 1) * 8, i = node0 + q;
          float f = 0.f;
          bool on = false;
          if (q < queries && sm.up[i] != -2) {
            if (x < kW) {
              on = x < r;
              if (on)
                f = lam_s[q * kLamPitch + fenwick_level(pos + sm.depth[i], (j << kLogW) + x)] *
                    expf(sm.after[x] + sm.first[i]);
            } else if (x - kW < N) {
              on = sm.above[i] >> (x - kW) & 1;
              if (on) f = wt[q * kNodes + x - kW];
            }
          }
          sc[t][u] = on ? f * sc[t][u] : 0.f;
        }
    }
    cp_async_wait<0>();
    consumer_sync();  // the keys and the tree's weights are done with, the values are there
    if (lane == 0) tc::mbar_arrive(&sm.empty[a.stages - 1]);
    if (mine) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < 4; u += 2) {
          uint32_t part[kPage];
          split2(sc[t][u], sc[t][u + 1], part);
          __nv_bfloat16* at = ps + (8 * t + lanes_i) * lay.tp + 16 * w + lanes_g + (u >> 1) * 8;
#pragma unroll
          for (int x = 0; x < kPage; ++x) {
            at[x * NQ * lay.tp] = __ushort_as_bfloat16((unsigned short)(part[x] & 0xffffu));
            at[x * NQ * lay.tp + lay.tp] = __ushort_as_bfloat16((unsigned short)(part[x] >> 16));
          }
        }
    }
    // values of nodes: none where a node is left out; infinities and NaN go by themselves, to the
    // nodes below them alone
    {
      const int rows = (N + 15) & ~15;
      bool odd = false;
      for (int x = tid; x < rows * (dv / 4); x += kConsumerThreads) {
        const int y = x / (dv / 4);
        T* p = vs + (kW + y) * lay.vp + 4 * (x - y * (dv / 4));
        if (y >= N || sm.up[y] == -2) {
#pragma unroll
          for (int u = 0; u < 4; ++u) p[u] = from_f32<T>(0.f);
        } else {
          const float4 v = load4(p);
          if (is_odd(v.x) || is_odd(v.y) || is_odd(v.z) || is_odd(v.w)) {
            odd = true;
            if (is_odd(v.x)) p[0] = from_f32<T>(0.f);
            if (is_odd(v.y)) p[1] = from_f32<T>(0.f);
            if (is_odd(v.z)) p[2] = from_f32<T>(0.f);
            if (is_odd(v.w)) p[3] = from_f32<T>(0.f);
          }
        }
      }
      if (odd) sm.odd = 1;
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
    consumer_sync();

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
      const T* gv = static_cast<const T*>(a.v) + row * a.sv[0] + h * a.sv[2];
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

    // the pages
    int st_ = 0, phase = 0;
    const int chunk = 4 * (ct & 1) + (lanes_g >> 1);
    const uint32_t off0 = tc::sw128_offset(lanes_i, chunk) + (lanes_g & 1) * 8;
    const uint32_t off1 = tc::sw128_offset(lanes_i + 1, chunk) + (lanes_g & 1) * 8;
    for (int x = 0; x < live && k0 < k1; ++x) {
      float part[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < 4; ++u) part[t][u] = 0.f;
      for (int d = k0; d < k1; d += span) {
        if (ok) ok = tc::mbar_wait_short(&sm.full[st_], phase);
        if (on) {
          const uint8_t* stage = dyn + (size_t)st_ * kStageBytes + (ct >> 1) * box_bytes;
          for (int y = 16 * kp; y < min(span, k1 - d); y += 16 * kparts) {
            const uint8_t* at = stage + (y >> box_log) * col_boxes * box_bytes + (y & (box_rows - 1)) * 128;
            const float2 x0 = *reinterpret_cast<const float2*>(at + off0), x1 = *reinterpret_cast<const float2*>(at + off1);
            const float2 x2 = *reinterpret_cast<const float2*>(at + off0 + 1024), x3 = *reinterpret_cast<const float2*>(at + off1 + 1024);
            uint32_t pa[kPage][4], p0[kPage], p1[kPage], p2[kPage], p3[kPage];
            split2(x0.x, x1.x, p0);
            split2(x0.y, x1.y, p1);
            split2(x2.x, x3.x, p2);
            split2(x2.y, x3.y, p3);
#pragma unroll
            for (int u = 0; u < kPage; ++u) {
              pa[u][0] = p0[u];
              pa[u][1] = p1[u];
              pa[u][2] = p2[u];
              pa[u][3] = p3[u];
            }
#pragma unroll
            for (int v = kIn - 1; v >= 0; --v) {
              uint32_t qb[NT][2];
              load_b<NT>(qb, qs + v * NQ * lay.kq, lay.kq, d + y);
#pragma unroll
              for (int u = kPage - 1; u >= 0; --u)
                if (u + v < kPage)
#pragma unroll
                  for (int t = 0; t < NT; ++t) mma_bf16(part[t], pa[u], qb[t][0], qb[t][1]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.empty[st_]);
        if (++st_ == a.stages) {
          st_ = 0;
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
      consumer_sync();  // the tokens' weights are done with
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

constexpr size_t kSmTwo = 115000, kSmOne = 232448;  // shared memory of a CTA where two are on an SM, and of one alone

template <typename T, int NT>
cudaError_t launch(const ll_cache& c, TreeArgs a, cudaStream_t s) {
  const int dk = (int)c.dk, dv = (int)c.dv;
  a.groups = (a.N + 8 * NT - 1) / (8 * NT);
  const int64_t items = (int64_t)a.n * c.H * a.groups;
  a.split = tree_split(items, dk, sm_count());
  const int share = ((dk + 15) / 16 + a.split - 1) / a.split * 16;
  a.box_log = share % 32 ? 4 : 5;
  const size_t body = (size_t)tree_layout<T, NT>(dk, dv, a.N).end + sizeof(TreeSmem) + 1024;
  size_t room = kSmTwo;
  if (body + 2 * kStageBytes > room) room = kSmOne;
  a.stages = (int)std::min<size_t>(kMaxTreeStages, (room - body) / kStageBytes);
  const size_t smem = (size_t)a.stages * kStageBytes + tree_layout<T, NT>(dk, dv, a.N).end;
  CUtensorMap pages;
  if (!make_pages_map(&pages, c.pages, c.n_pages, c.H, c.dk, c.dv, 1 << a.box_log)) return cudaErrorInvalidValue;
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
