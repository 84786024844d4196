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
  int split_log, groups_log;    // CTAs of a cluster, groups of nodes
  int own, stages, box_rows;    // stages that are only the ring's, all of them; rows of a stage
  FastDiv heads, per_qk;        // H, H / Hqk
};

// A CTA serves one (row, head) for up to 8 NT nodes: eight warps that compute, and one that
// keeps a ring of stages of up to 16 KB of the pages filled.  The products run on the tensor cores
// as out^T = page^T q^T: a page's values go from the ring to the fragments as they are, and the nodes
// are the narrow side.  mma.sync, not tcgen05: a page lies in memory with the output's
// columns side by side, and every value of it is used for at most 64 nodes, so HBM and, with small
// trees, the instructions around the products are the bounds, not the tensor pipe.
//
// Precision.  bf16 outputs are the fp32 ones, rounded once.  q, k and v of a bf16 cache enter their products as they are,
// a page's value as three bf16 parts that together are the fp32 value, and a token's weight as two tf32 parts
// that leave 2^-22.  (Pages and weights rounded to tf32 for bf16 outputs took 77 and 119 us where this takes 88 and 154, and
// moved the outputs by up to 2^-11 of each product; pages as two tf32 parts, 108 and 176.)  With fp32 tokens everything
// is two tf32 parts, and all four products of them are taken: the first parts are cut off towards zero, so the fourth
// is of one sign and adds up.  The three with a second part are summed apart from the first (rel-L2 of the outputs
// 3.3e-7 for the batch below in fp32, 1.1e-6 in one sum; 2.3e-7 in fp32 multiply-adds).  All sums are fp32, and a page is
// summed by itself before it is weighted per node.
//
// Measured (GB300, calls in a row; floor: the bytes at the measured copy rate of 6.7 TB/s).  One sequence, 16 heads, d
// 128, 8 nodes, position 12345: 9.3 us, a chain of latencies (inputs, scores, weights, values, pages, two cluster
// barriers).  61 sequences of such heads at 0..16383, up to 32 nodes: 88 us, 3.5 TB/s, floor 45.  24 sequences of
// 48 heads on one q/k head, dv 64, 64 nodes, 4096..131071: 154 us, 1.6 TB/s, floor 36.  There a page's third part is 17 us
// and a weight's second one 16; registers and the weights' room allow two CTAs per SM (18 warps; 40 % of the issue slots,
// tensor pipe 27 %), which hide the part before the pages only partly: one stage of pages is on its way in it, and none in
// the batch's.  fp32 tokens, of which a CTA per SM fits above 16 nodes: the batch 209 us, its trees of 48 nodes, which pass the
// pages twice, 393 us, the shared heads 367 us (floors 52, 56, 39).
constexpr int kTreeWarps = 8, kConsumers = 32 * kTreeWarps, kTreeThreads = kConsumers + 32;
constexpr int kFiller = kTreeWarps;    // the warp that fills the ring
constexpr int kWalkers = kTreeWarps - 2;  // the first of the two warps that have a node per thread
constexpr int kStageBytes = 16384;
constexpr int kMaxTreeStages = 8;
constexpr int kTreeSplit = 8;          // CTAs of a cluster
constexpr int kQPitch = 132;           // floats from query to query, of fp32 tokens
constexpr int kPairPitch = 136;        // and bf16 ones, of bf16 tokens

template <typename T>
struct Parts {
  static constexpr int in = sizeof(T) == 2 ? 1 : 2;  // of tokens, in tf32
};
__host__ __device__ constexpr int pad4(int x) { return (x + 3) & ~3; }

// Shared memory behind the ring's own stages, in bytes.  The tokens' weights and values are done with
// before the pages: whole stages of their place then join the ring.
struct TreeLayout {
  int vp, tp, lp;             // elements from row to row: v, the tokens' weights, lambda
  int p, v, q, lam, pw, end;  // where each begins
};
template <typename T, int NT>
__host__ __device__ __forceinline__ TreeLayout tree_layout(int dv, int N, int M) {
  const int dv16 = (dv + 15) & ~15, tokens = kW + ((N + 15) & ~15);
  TreeLayout l;
  l.vp = dv16 + (sizeof(T) == 2 ? 8 : 4);  // rows 2 i and 2 i + 1 of four threads fall into banks of their own
  l.tp = tokens + 8;
  l.lp = pad4(M + kLogW + 1);
  l.p = 0;
  l.v = l.p + 8 * NT * l.tp * 4;
  l.q = l.v + tokens * l.vp * (int)sizeof(T);
  l.lam = l.q + 8 * NT * (sizeof(T) == 2 ? kPairPitch * 2 : 2 * kQPitch * 4);
  l.pw = l.lam + (NT == 8 ? 8 * NT * l.lp * 4 : 0);  // (up to 32 nodes: with the tree's decays)
  l.end = l.pw + M * 8 * NT * 4;
  return l;
}

// CTAs that registers leave on an SM.
template <typename T, int NT>
constexpr int tree_ctas() { return sizeof(T) == 2 ? (NT <= 4 ? 3 : 2) : NT <= 2 ? 2 : 1; }

struct TreeSmem {
  uint64_t full[kMaxTreeStages], empty[kMaxTreeStages];
  float after[kW];                   // log decay from each token of the block to the context's last
  float first[kNodes];               // log decay of the path to each node
  float page_log[kMaxLevels];        // the live pages, lowest level first
  int page_at[kMaxLevels], page_lv[kMaxLevels];
  unsigned long long above[kNodes];  // nodes on the path, itself included
  float since;
  unsigned bad[kTreeWarps + 1];      // what each warp found
  int odd;                           // a node's v has infinities or NaN
  signed char up[kNodes], depth[kNodes];
};

// Of the eight warps that compute, and of the two that have the nodes.
__device__ __forceinline__ void consumer_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kConsumers) : "memory"); }
__device__ __forceinline__ void walkers_sync() { asm volatile("barrier.cta.sync 2, 64;" ::: "memory"); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
__device__ __forceinline__ void load2(float2& v, uint32_t at) {
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x to the nearest tf32 (half up: carries into the exponent as they should, infinities stay).
__device__ __forceinline__ uint32_t tf32_of(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
// x as two tf32 parts.  The first is cut off towards zero, and what is left of a value that is not 0 is never
// 0 or NaN (infinity less itself) but at least the least normal value: then infinities come out as in
// the sum itself.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  const float rest = fmaxf(fabsf(x) - fabsf(__uint_as_float(hi)), fminf(fabsf(x), 0x1p-126f));
  lo = tf32_of(rest) | (hi & 0x80000000u);
}
// The leading 8 bits of x and y, as bf16; they keep the rest, so that three such parts are the fp32 value itself.
// (Infinities leave NaN.)
__device__ __forceinline__ uint32_t lead_bf16(float& x, float& y) {
  const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
  x -= __uint_as_float(a & 0xffff0000u);
  y -= __uint_as_float(b & 0xffff0000u);
  return __byte_perm(a, b, 0x7632);
}
// The products with a second part are summed apart: the tensor cores cut a sum off at its own size, towards zero, and
// would lose most of them, all of one sign, behind the products of the first parts.
template <int NT>
__device__ __forceinline__ void add_parts(float (&sum)[NT][4], const float (&low)[NT][4]) {
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int u = 0; u < 4; ++u) sum[t][u] += low[t][u];
}
// Two neighbouring values as tf32 parts.
__device__ __forceinline__ void parts2(const __nv_bfloat16* p, uint32_t (&part)[1][2]) {
  const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
  part[0][0] = x << 16;
  part[0][1] = x & 0xffff0000u;
}
__device__ __forceinline__ void parts2(const float* p, uint32_t (&part)[2][2]) {
  const float2 x = *reinterpret_cast<const float2*>(p);
  split_tf32(x.x, part[0][0], part[1][0]);
  split_tf32(x.y, part[0][1], part[1][1]);
}

// 8 values of a row from column k on, 0 past `width`, as they are.
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* row, int k, int width, bool vec) {
  uint4 x = make_uint4(0u, 0u, 0u, 0u);
  if (vec) {
    if (k < width) x = *reinterpret_cast<const uint4*>(row + k);
  } else {
    uint32_t* w = &x.x;
#pragma unroll 1
    for (int u = 0; u < 8; ++u)
      if (k + u < width) {
        const uint32_t e = (uint32_t)__bfloat16_as_ushort(row[k + u]) << (u & 1) * 16;
        if (u < 2) w[0] |= e;
        else if (u < 4) w[1] |= e;
        else if (u < 6) w[2] |= e;
        else w[3] |= e;
      }
  }
  return x;
}
struct Float8 {
  float e[8];
};
__device__ __forceinline__ Float8 load8(const float* row, int k, int width, bool vec) {
  Float8 x;
  if (vec) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 a = k < width ? *reinterpret_cast<const float4*>(row + k) : z;
    const float4 b = k + 4 < width ? *reinterpret_cast<const float4*>(row + k + 4) : z;
    x.e[0] = a.x; x.e[1] = a.y; x.e[2] = a.z; x.e[3] = a.w;
    x.e[4] = b.x; x.e[5] = b.y; x.e[6] = b.z; x.e[7] = b.w;
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u) x.e[u] = k + u < width ? row[k + u] : 0.f;
  }
  return x;
}
// As tf32 parts: part[p][u] of value u.
__device__ __forceinline__ void parts_of(const Float8& x, uint32_t (&part)[2][8]) {
#pragma unroll
  for (int u = 0; u < 8; ++u) split_tf32(x.e[u], part[0][u], part[1][u]);
}

template <typename T>
__device__ __forceinline__ bool whole_pieces(const T* p, int64_t stride, int width) {
  return ((width | stride) * sizeof(T)) % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}
// Rows to shared memory by the consumers, asynchronously where they are whole 16-byte pieces.
template <typename T>
__device__ __forceinline__ void bring_rows(T* dst, int pitch, const T* src, int64_t stride, int rows, int width) {
  if (whole_pieces(src, stride, width)) {
    constexpr int kPieces = 8 * (int)sizeof(T), kStep = kConsumers / kPieces;  // 16-byte pieces of 128 columns
    const int y = threadIdx.x / kPieces, x = (threadIdx.x & (kPieces - 1)) * (16 / (int)sizeof(T));
    if (x >= width) return;
    uint32_t to = tc::smem_u32(dst + y * pitch + x);
    const T* from = src + y * stride + x;
    for (int r = y; r < rows; r += kStep, to += kStep * pitch * (int)sizeof(T), from += kStep * stride) cp_async16(to, from);
  } else {
    const int x = threadIdx.x & 127;
    if (x < width)
      for (int r = threadIdx.x >> 7; r < rows; r += kConsumers >> 7) dst[r * pitch + x] = src[r * stride + x];
  }
}

// Infinity or NaN, in x or in either half of two bf16.
__device__ __forceinline__ bool is_odd(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }
template <typename T>
__device__ __forceinline__ bool is_odd_word(uint32_t x) {
  return (sizeof(T) == 2 && (x & 0x7f80u) == 0x7f80u) || (x & 0x7f800000u) == 0x7f800000u;
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
    cache_tree_kernel(const __grid_constant__ CUtensorMap pages, const __grid_constant__ ll_cache c,
                      const __grid_constant__ TreeArgs a) {
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ TreeSmem sm;
  constexpr int kIn = Parts<T>::in, NQ = 8 * NT;
  const int H = (int)c.H, dk = (int)c.dk, dv = (int)c.dv, M = (int)c.levels;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int Z = 1 << a.split_log, sp = blockIdx.x & (Z - 1), item = blockIdx.x >> a.split_log;
  const int node0 = (item & ((1 << a.groups_log) - 1)) * NQ, rh = item >> a.groups_log;
  const int row = rh / a.heads, h = rh - row * H, hq = h / a.per_qk;
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
  const int64_t first_node = (int64_t)row * a.N;
  uint8_t* body = dyn + a.own * kStageBytes;
  const TreeLayout lay = tree_layout<T, NT>(dv, a.N, M);
  float* ps = reinterpret_cast<float*>(body + lay.p);  // [NQ][lay.tp]
  T* vs = reinterpret_cast<T*>(body + lay.v);
  float* qs = reinterpret_cast<float*>(body + lay.q);  // fp32 tokens: [parts][NQ][kQPitch]; of every 8 columns the even ones, then the odd ones
  __nv_bfloat16* qb = reinterpret_cast<__nv_bfloat16*>(body + lay.q);  // bf16 tokens: [NQ][kPairPitch]
  float* page_w = reinterpret_cast<float*>(body + lay.pw);
  float* wt = reinterpret_cast<float*>(dyn + (a.own - 1) * kStageBytes);  // log decays of the tree, in the last own stage until the pages need it
  float* lam_s = NT == 8 ? reinterpret_cast<float*>(body + lay.lam) : wt + NQ * kNodes;
  float* la_s = ps;                                                          // the nodes' log a, until their weights are there
  float* red = reinterpret_cast<float*>(dyn);                               // the ring, behind the pages

  // geometry of the pages: col_boxes boxes of 32 columns, the rows in stages of box_rows
  const int col_boxes = (dv + 31) / 32, box_rows = a.box_rows, box_bytes = box_rows * 128;
  const int share = (((dk + 15) / 16 + Z - 1) >> a.split_log) * 16;
  const int k0 = min(dk, sp * share), k1 = min(dk, k0 + share);  // this CTA's rows
  // the filler's place in the pages: page, row; stage and how often it was used
  int m = 0, d0 = k0, st = 0, use = 0;
  auto bring_stage = [&]() {
    tc::mbar_arrive_expect_tx(&sm.full[st], col_boxes * box_bytes);
    for (int x = 0; x < col_boxes; ++x)
      tc::tma_load_4d(&pages, &sm.full[st], dyn + st * kStageBytes + x * box_bytes, 32 * x, d0, h, sm.page_at[m]);
    if ((d0 += box_rows) >= k1) {
      d0 = k0;
      ++m;
    }
    if (++st == a.stages) {
      st = 0;
      ++use;
    }
  };
  const T* gv = static_cast<const T*>(a.v) + row * a.sv[0] + h * a.sv[2];
  const T* wv = static_cast<const T*>(c.win_v) + ((int64_t)s * H + h) * kW * dv;
  const int lanes_g = lane >> 2, lanes_i = 2 * (lane & 3);
  const int tiles = kW / 16 + (N + 15) / 16;  // of 16 tokens: the block's, then the nodes; one per warp
  const bool mine = w < tiles && (w & (Z - 1)) == sp && (w >= kW / 16 || 16 * w < r);
  // the last two warps have a node per thread: their tiles are there for most nodes only
  const int node = w >= kWalkers && w < kTreeWarps ? tid - 32 * kWalkers : -1;
  bool ok = true;
  float sc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int u = 0; u < 4; ++u) sc[t][u] = 0.f;

  // everything that is read, first
  if (w == kFiller) {
    const bool here = lane < M && (j >> lane) & 1;
    const int e = here ? c.page_table[(int64_t)s * M + lane] : 0;
    const float log = here ? c.page_log[(((int64_t)s * 2 + par) * M + lane) * H + h] : 0.f;
    const bool before = before_pages(c, s, pos);
    if (lane == 0) {
      for (int i = 0; i < a.stages; ++i) {
        tc::mbar_init(&sm.full[i], 1);
        tc::mbar_init(&sm.empty[i], kTreeWarps);
      }
      tc::fence_mbar_init();
      sm.odd = 0;
    }
    if (here) {
      const int at = __popc(j & ((1 << lane) - 1));
      sm.page_at[at] = e;
      sm.page_lv[at] = lane;
      sm.page_log[at] = log;
    }
    const bool missing = __any_sync(0xffffffffu, e < 0 || e >= c.n_pages);
    __syncwarp();
    if (lane == 0) {
      sm.bad[w] = (missing ? LL_CACHE_ERR_MISSING : 0) | (before ? LL_CACHE_ERR_POSITION : 0);
      if (!missing && k0 < k1)
        while (m < live && use == 0 && st < a.own - 1) bring_stage();
    }
    __syncthreads();
  } else {
    int up = -2;
    float la = 0.f;
    if (node >= 0 && node < a.N) {
      up = a.parents[first_node + node];
      if (a.log_a) la = a.log_a[(first_node + node) * H + h];
    }
    const T* gk = static_cast<const T*>(a.k) + row * a.sk[0] + hq * a.sk[2];
    const T* wk = static_cast<const T*>(c.win_k) + ((int64_t)s * (int)c.Hqk + hq) * kW * dk;
    const bool key_vec = w < kW / 16 ? whole_pieces(wk, dk, dk) : whole_pieces(gk, a.sk[1], dk);
    // the thread's keys: tokens g and g + 8 of its warp's tile, of every 32 columns 8 neighbouring ones
    const T* key[2];
    int key_width[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = 16 * w + lanes_g + 8 * u;
      key[u] = x < kW ? wk + x * dk : gk + (x - kW) * a.sk[1];
      key_width[u] = mine && (x < kW ? x < r : x - kW < N) ? dk : 0;
    }
    decltype(load8(key[0], 0, 0, true)) key_e[sizeof(T) == 2 ? 4 : 1][2];  // (fp32: brought when they are needed)
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int u = 0; u < 2; ++u) key_e[d][u] = load8(key[u], 32 * d + 4 * lanes_i, key_width[u], key_vec);
    }
    for (int q = w; q < queries; q += kTreeWarps)
      if (lane < M + kLogW + 1)
        tc::cp_async4(lam_s + q * lay.lp + lane, a.lam + ((first_node + node0 + q) * H + h) * a.L + lane, 4);
    if (node < 0) {
      const T* gq = static_cast<const T*>(a.q) + row * a.sq[0] + hq * a.sq[2] + node0 * a.sq[1];
      const bool vec = whole_pieces(gq, a.sq[1], dk);
      const int k = (tid & 15) * 8;
      if (k < ((dk + 31) & ~31))
        for (int q = tid >> 4; q < (sizeof(T) == 2 ? NQ : queries); q += 2 * kWalkers) {
          if constexpr (sizeof(T) == 2) {
            // (0 behind the last: what stands there would make NaN, and those are summed once more)
            *reinterpret_cast<uint4*>(qb + q * kPairPitch + k) = load8(gq + q * a.sq[1], k, q < queries ? dk : 0, vec);
          } else {
            uint32_t part[2][8];
            parts_of(load8(gq + q * a.sq[1], k, dk, vec), part);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint4* to_ = reinterpret_cast<uint4*>(qs + (y * NQ + q) * kQPitch + k);
              to_[0] = make_uint4(part[y][0], part[y][2], part[y][4], part[y][6]);
              to_[1] = make_uint4(part[y][1], part[y][3], part[y][5], part[y][7]);
            }
          }
        }
    }
    cp_async_commit();  // lambda first
    bring_rows(vs, lay.vp, wv, dv, r, dv);
    bring_rows(vs + kW * lay.vp, lay.vp, gv, a.sv[1], N, dv);
    cp_async_commit();
    {
      unsigned bad = 0;
      if (node >= 0) {  // the nodes' paths, and the log decays along those of the queries
        const bool fine = up < node && up >= -2;
        up = fine ? up : -2;
        sm.up[node] = (signed char)up;
        la_s[node] = up != -2 ? la : 0.f;
        walkers_sync();
        if (!fine) bad = LL_CACHE_ERR_TREE;
        unsigned long long above = 0;
        int depth = -1;
        const int q = node - node0;
        const bool asks = q >= 0 && q < queries;
        float acc = 0.f;  // log a behind x up to the node
        for (int x = up == -2 ? -1 : node; x >= 0; x = sm.up[x]) {
          above |= 1ull << x;
          ++depth;
          if (sm.up[x] == -2) bad = LL_CACHE_ERR_TREE;  // a child of a node that is left out
          if (asks) wt[q * kNodes + x] = acc;
          acc += la_s[x];
        }
        sm.first[node] = acc;
        sm.above[node] = above;
        sm.depth[node] = (signed char)depth;
        if (depth >= 0 && !position_ok(c, pos + depth)) bad |= LL_CACHE_ERR_POSITION;
      } else if (w == 0) {
        float since;
        block_decays(c.win_log_a + ((int64_t)s * H + h) * kW, r, c.page_from[s * 2 + par], sm.after, &since);
        if (lane == 0) sm.since = since;
      }
      bad = __reduce_or_sync(0xffffffffu, bad);
      if (lane == 0) sm.bad[w] = bad;
    }
    cp_async_wait<1>();
    __syncthreads();

    // scores of 16 tokens per warp, K q^T, not yet weighted.  Of 32 columns each thread has 8 neighbouring ones of
    // two keys, and takes those of its query: which column stands where in a product does not matter
    if (mine) {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if (32 * d >= dk) break;
        if constexpr (sizeof(T) == 2) {
          const uint4 k0_ = key_e[d][0], k1_ = key_e[d][1];
          const uint32_t ka[2][4] = {{k0_.x, k1_.x, k0_.y, k1_.y}, {k0_.z, k1_.z, k0_.w, k1_.w}};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 q = *reinterpret_cast<const uint4*>(qb + (8 * t + lanes_g) * kPairPitch + 32 * d + 4 * lanes_i);
            mma_bf16(sc[t], ka[0], q.x, q.y);
            mma_bf16(sc[t], ka[1], q.z, q.w);
          }
        } else {
          float low[NT][4] = {};
          uint32_t ka[2][2][8];
#pragma unroll
          for (int u = 0; u < 2; ++u) parts_of(load8(key[u], 32 * d + 4 * lanes_i, key_width[u], key_vec), ka[u]);
#pragma unroll
          for (int y = 1; y >= 0; --y)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint4* q = reinterpret_cast<const uint4*>(qs + (y * NQ + 8 * t + lanes_g) * kQPitch + 32 * d + 4 * lanes_i);
              const uint4 even = q[0], odd = q[1];
#pragma unroll
              for (int x = 1; x >= 0; --x) {
                float(&f)[4] = x + y ? low[t] : sc[t];
                mma_tf32(f, ka[0][x][0], ka[1][x][0], ka[0][x][1], ka[1][x][1], even.x, odd.x);
                mma_tf32(f, ka[0][x][2], ka[1][x][2], ka[0][x][3], ka[1][x][3], even.y, odd.y);
                mma_tf32(f, ka[0][x][4], ka[1][x][4], ka[0][x][5], ka[1][x][5], even.z, odd.z);
                mma_tf32(f, ka[0][x][6], ka[1][x][6], ka[0][x][7], ka[1][x][7], even.w, odd.w);
              }
            }
          add_parts(sc, low);
        }
      }
    }
  }
  unsigned bad = 0;
#pragma unroll
  for (int i = 0; i <= kTreeWarps; ++i) bad |= sm.bad[i];
  if (bad) {
    if (tid == 0 && speaks) raise(c, bad);
    if (w == kFiller && lane == 0)  // the copies on their way
      for (int i = 0; i < st; ++i) tc::mbar_wait_short(&sm.full[i], 0);
    tc::cp_async_wait_all();
    return;
  }

  if (w == kFiller) {
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
    if (Z > 1) {
      cluster_arrive();
      cluster_wait();
      cluster_arrive();
      cluster_wait();
    }
  } else {
    // the weighted scores
    if (mine) {
      const bool nodes = w >= kW / 16;
      const int x0 = 16 * w + lanes_g - (nodes ? kW : 0);  // the thread's tokens: x0 and x0 + 8
      // where they stand
      const int s0 = nodes ? pos + sm.depth[x0] : (j << kLogW) + x0, s1 = nodes ? pos + sm.depth[x0 + 8] : s0 + 8;
      const float after0 = nodes ? 0.f : sm.after[x0], after1 = nodes ? 0.f : sm.after[x0 + 8];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int q = 8 * t + lanes_i;
        float f[2][2];  // [node q, q + 1][token x0, x0 + 8]
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int depth = sm.depth[node0 + q + u], tq = pos + depth;
          const float* lam = lam_s + (q + u) * lay.lp;
          if (nodes) {
            const unsigned long long up = sm.above[node0 + q + u] >> x0;
            const float* log = wt + (q + u) * kNodes + x0;
            f[u][0] = up & 1 ? lam[fenwick_level(tq, s0)] * expf(log[0]) * sc[t][u] : 0.f;
            f[u][1] = up >> 8 & 1 ? lam[fenwick_level(tq, s1)] * expf(log[8]) * sc[t][2 + u] : 0.f;
          } else {
            const float first = sm.first[node0 + q + u];
            f[u][0] = depth >= 0 && s0 < pos ? lam[fenwick_level(tq, s0)] * expf(after0 + first) * sc[t][u] : 0.f;
            f[u][1] = depth >= 0 && s1 < pos ? lam[fenwick_level(tq, s1)] * expf(after1 + first) * sc[t][2 + u] : 0.f;
          }
        }
        float* at = ps + q * lay.tp + 16 * w + lanes_g;
#pragma unroll
        for (int u = 0; u < 4; ++u) at[(u & 1) * lay.tp + (u >> 1) * 8] = f[u & 1][u >> 1];
      }
    }
    for (int x = tid; x < live * NQ; x += kConsumers) {
      const int y = x / NQ, q = x - y * NQ, depth = sm.depth[node0 + q];
      float f = 0.f;
      if (depth >= 0) {
        const int lv = (pos + depth) >> kLogW > j ? max(sm.page_lv[y], to) : sm.page_lv[y];
        f = lam_s[q * lay.lp + kLogW + 1 + lv] * expf(sm.page_log[y] + sm.since + sm.first[node0 + q]);
      }
      page_w[x] = f;
    }
    // the values.  Behind the block's tokens and the nodes, and where a node is left out: 0.  Infinities
    // and NaN of a node go by themselves, to the nodes below it alone; in the products an infinity is the least normal value
    // of its sign (an infinite weight makes the sum's infinity of that, where 0 would make NaN), NaN is 0
    tc::cp_async_wait_all();
    {
      constexpr int kWords = 8 * (int)sizeof(T);  // 16-byte pieces that 128 columns have
      const int piece = tid & (kWords - 1), words = min(4, (dv * (int)sizeof(T) - 16 * piece) / 4);
      if (words > 0) {
        for (int y = r + tid / kWords; y < ((r + 15) & ~15); y += kConsumers / kWords)
          reinterpret_cast<uint4*>(vs + y * lay.vp)[piece] = make_uint4(0u, 0u, 0u, 0u);
        for (int y = tid / kWords; y < ((N + 15) & ~15); y += kConsumers / kWords) {
          uint32_t* p = reinterpret_cast<uint32_t*>(vs + (kW + y) * lay.vp) + 4 * piece;
          if (y >= N || sm.up[y] == -2) {
            *reinterpret_cast<uint4*>(p) = make_uint4(0u, 0u, 0u, 0u);
          } else {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            if (is_odd_word<T>(v.x) || is_odd_word<T>(v.y) || (words > 2 && (is_odd_word<T>(v.z) || is_odd_word<T>(v.w)))) {
              sm.odd = 1;
              T* e = reinterpret_cast<T*>(p);
#pragma unroll 1
              for (int u = 0; u < words * 4 / (int)sizeof(T); ++u)
                if (const float f = to_f32(e[u]); is_odd(f)) e[u] = from_f32<T>(f != f ? 0.f : copysignf(0x1p-126f, f));
            }
          }
        }
      }
    }
    tc::fence_proxy_async_smem();  // the pages are written behind what the last own stage holds
    consumer_sync();  // the tokens' weights and values are there, the tree's decays are done with
    if (lane == 0) tc::mbar_arrive(&sm.empty[a.own - 1]);

    // a warp's 16 columns; where there are few, warps share them by tokens and by rows of the pages
    const int cols = (dv + 15) / 16, wide_log = cols > 4 ? 3 : cols > 2 ? 2 : cols - 1, wide = 1 << wide_log;
    const int ct = w & (wide - 1), kp = w >> wide_log, kparts = kTreeWarps >> wide_log;
    const bool on = ct < cols;
    const int col = 16 * ct + 2 * lanes_g;  // the thread's columns: this one and the next
    float acc[NT][4];                       // [node tile][column, node: (0, 0), (0, 1), (1, 0), (1, 1)]
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int u = 0; u < 4; ++u) acc[t][u] = 0.f;
    if (on) {
      int turn = 0;
      float low[kIn == 2 ? NT : 1][4] = {};
      for (int tile = sp; tile < tiles; tile += Z) {
        if (tile < kW / 16 && 16 * tile >= r) continue;
        if ((turn++ & (kparts - 1)) != kp) continue;
#pragma unroll
        for (int y = 0; y < 2; ++y) {  // 8 tokens: 2 i and 2 i + 1 of each thread
          const T* v0 = vs + (16 * tile + 8 * y + lanes_i) * lay.vp + col;
          uint32_t va[kIn][2], vb[kIn][2];  // tokens 2 i and 2 i + 1
          parts2(v0, va);
          parts2(v0 + lay.vp, vb);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            uint32_t p[2][2];
            parts2(ps + (8 * t + lanes_g) * lay.tp + 16 * tile + 8 * y + lanes_i, p);
#pragma unroll
            for (int x = 1; x >= 0; --x)
#pragma unroll
              for (int i = kIn - 1; i >= 0; --i)
                mma_tf32(kIn == 2 && x + i ? low[kIn == 2 ? t : 0] : acc[t], va[i][0], va[i][1], vb[i][0], vb[i][1], p[x][0], p[x][1]);
          }
        }
      }
      if constexpr (kIn == 2) add_parts(acc, low);
    }
    if (sm.odd && on && kp == 0 && col < dv) {
#pragma unroll 1
      for (int y = 0; y < N; ++y) {
        if (((kW + y) / 16 & (Z - 1)) != sp) continue;
        const float v0 = to_f32(gv[y * a.sv[1] + col]), v1 = to_f32(gv[y * a.sv[1] + col + 1]);
        if (!is_odd(v0) && !is_odd(v1)) continue;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int q = 8 * t + lanes_i + (u & 1);
            const float v = u >> 1 ? v1 : v0;
            if (q >= queries || !(sm.above[node0 + q] >> y & 1) || !is_odd(v)) continue;
            acc[t][u] = fmaf(ps[q * lay.tp + kW + y], v, acc[t][u]);
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
    // a column tile); a step's 16 rows are 2 i, 2 i + 1, 2 i + 8 and 2 i + 9 of each thread, which keeps the reads
    // free of conflicts under the swizzle.  Two columns of two rows are a fragment as they come.
    if (k0 < k1) {
      const int chunk = 4 * (ct & 1) + (lanes_g >> 1), first_row = 16 * (wide > 1 ? 2 * kp : kp);
      const uint32_t rows_at = tc::smem_u32(dyn) + (ct >> 1) * box_bytes + (lanes_g & 1) * 8 + 128 * first_row;
      const uint32_t off0 = rows_at + tc::sw128_offset(lanes_i, chunk), off1 = rows_at + tc::sw128_offset(lanes_i + 1, chunk);
      // bf16: a step's 16 columns of two node tiles (of one, twice); fp32: 16 columns of a part of one
      const uint32_t q_at = sizeof(T) == 2
          ? tc::smem_u32(qb) + (((lane & 7) + (NT > 1 ? (lane >> 4) * 8 : 0)) * kPairPitch + (lane >> 3 & 1) * 8 + first_row) * 2
          : tc::smem_u32(qs) + (lane & 7) * kQPitch * 4 + (lane >> 3) * 16 + 4 * first_row;
      int stage = 0, phase = 0;
      for (int x = 0; x < live; ++x) {
        float part[NT][4] = {}, low[kIn == 2 ? NT : 1][4] = {};
        for (int d = k0; d < k1; d += box_rows) {
          if (ok) ok = tc::mbar_wait_short(&sm.full[stage], phase);
          const uint32_t at0 = off0 + stage * kStageBytes, at1 = off1 + stage * kStageBytes, q = q_at + (int)sizeof(T) * d;
          const int rows = min(box_rows, k1 - d) - first_row;  // from this warp's first on
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            if (!on || 16 * z >= rows || (z && wide == 1)) continue;
            float2 v[4];
            load2(v[0], at0 + 2048 * z);
            load2(v[1], at1 + 2048 * z);
            load2(v[2], at0 + 2048 * z + 1024);
            load2(v[3], at1 + 2048 * z + 1024);
            if constexpr (sizeof(T) == 2) {
              uint32_t pa[3][4];
#pragma unroll
              for (int u = 0; u < 3; ++u) {
                pa[u][0] = lead_bf16(v[0].x, v[1].x);
                pa[u][1] = lead_bf16(v[0].y, v[1].y);
                pa[u][2] = lead_bf16(v[2].x, v[3].x);
                pa[u][3] = lead_bf16(v[2].y, v[3].y);
              }
#pragma unroll
              for (int t = 0; t < NT; t += 2) {
                uint32_t b[4];
                ldmatrix4(b[0], b[1], b[2], b[3], q + (8 * t * kPairPitch + 16 * z) * 2);
#pragma unroll
                for (int u = 2; u >= 0; --u) {
                  mma_bf16(part[t], pa[u], b[0], b[1]);
                  if (NT > 1) mma_bf16(part[t + (NT > 1)], pa[u], b[2], b[3]);
                }
              }
            } else {
              uint32_t pa[2][8];
#pragma unroll
              for (int u = 0; u < 8; ++u) split_tf32(u & 1 ? v[u >> 1].y : v[u >> 1].x, pa[0][u], pa[1][u]);
#pragma unroll
              for (int y = 1; y >= 0; --y)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                  uint32_t b[4];
                  ldmatrix4(b[0], b[1], b[2], b[3], q + ((y * NQ + 8 * t) * kQPitch + 16 * z) * 4);
#pragma unroll
                  for (int u = 1; u >= 0; --u) {
                    float(&f)[4] = u + y ? low[t] : part[t];
                    mma_tf32(f, pa[u][0], pa[u][1], pa[u][2], pa[u][3], b[0], b[1]);
                    mma_tf32(f, pa[u][4], pa[u][5], pa[u][6], pa[u][7], b[2], b[3]);
                  }
                }
            }
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.empty[stage]);
          if (++stage == a.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if constexpr (sizeof(T) == 2) {
          // NaN: of the sum itself, or of an infinity's parts.  The sums that have it once more, value by value
          bool nan = false;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int u = 0; u < 4; ++u) nan |= part[t][u] != part[t][u];
          if (nan && on && col < dv) {
            unsigned which = 0;
#pragma unroll
            for (int e = 0; e < 4 * NT; ++e)
              if (part[e >> 2][e & 3] != part[e >> 2][e & 3] && sm.depth[node0 + 8 * (e >> 2) + lanes_i + (e & 1)] >= 0) which |= 1u << e;
            const float* page = c.pages + ((int64_t)sm.page_at[x] * H + h) * dk * dv + col;
#pragma unroll 1
            for (; which; which &= which - 1) {
              const int e = __ffs(which) - 1;
              const __nv_bfloat16* qr = qb + (8 * (e >> 2) + lanes_i + (e & 1)) * kPairPitch;
              float f = 0.f;
#pragma unroll 1
              for (int d = k0; d < k1; d += box_rows)
#pragma unroll 1
                for (int y = first_row; f == f && y < min(min(box_rows, k1 - d), first_row + (wide > 1 ? 32 : 16)); ++y)
                  f = fmaf(page[(int64_t)(d + y) * dv + (e >> 1 & 1)], __bfloat162float(qr[d + y]), f);
#pragma unroll
              for (int i = 0; i < 4 * NT; ++i)
                if (i == e) part[i >> 2][i & 3] = f;
            }
          }
          __syncwarp();
        } else {
          add_parts(part, low);
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
    }
    if (!ok && lane == 0) raise(c, LL_CACHE_ERR_WAIT);

    // sums over the warps that share columns, and over the cluster
    const bool pairs = (reinterpret_cast<uintptr_t>(a.out) & (a.out_f32 ? 7u : 3u)) == 0;
    const int64_t out_at = ((first_node + node0) * H + h) * dv;
    auto put = [&](int t, int tile, const float (&x)[4]) {  // of 16 columns
      const int col_ = 16 * tile + 2 * lanes_g;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int q = 8 * t + lanes_i + u;
        if (col_ >= dv || sm.depth[node0 + q] < 0) continue;
        const int64_t at = out_at + (int64_t)q * H * dv + col_;
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
      return;
    }
    consumer_sync();  // the ring is done with: [column tile][node tile][warp of the rows][thread]
#pragma unroll
    for (int t = 0; t < NT; ++t)
      *reinterpret_cast<float4*>(red + (((ct * NT + t) * kparts + kp) * 32 + lane) * 4) =
          make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    const int sums = NT * wide;
    if (Z == 1) {
      consumer_sync();
#pragma unroll 1
      for (int x = w; x < sums; x += kTreeWarps) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < kparts; ++p) y = add4(y, *reinterpret_cast<const float4*>(red + ((x * kparts + p) * 32 + lane) * 4));
        const float z[4] = {y.x, y.y, y.z, y.w};
        put(x & (NT - 1), x / NT, z);
      }
    } else {
      cluster_arrive();
      cluster_wait();
#pragma unroll 1
      for (int x = w * Z + sp; x < sums; x += kTreeWarps * Z) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int z = 0; z < Z; ++z)
          for (int p = 0; p < kparts; ++p) y = add4(y, load_remote4(red + ((x * kparts + p) * 32 + lane) * 4, z));
        const float z[4] = {y.x, y.y, y.z, y.w};
        put(x & (NT - 1), x / NT, z);
      }
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    }
  }
}

// CTAs per item: doubled while that leaves the launch within the SMs, each with at least 16 rows of the pages.
int tree_split_log(int64_t items, int dk, int sms) {
  int log = 0;
  while (1 << log < kTreeSplit && (items << (log + 1)) <= sms && dk > 16 << log) ++log;
  return log;
}

constexpr size_t kSm = 233472;  // shared memory of an SM

template <typename T, int NT>
cudaError_t launch(const ll_cache& c, TreeArgs a, cudaStream_t s) {
  const int dk = (int)c.dk, dv = (int)c.dv;
  a.groups_log = a.N > 8 * NT ? 1 : 0;
  const int64_t items = (int64_t)a.n * c.H << a.groups_log;
  a.split_log = tree_split_log(items, dk, sm_count());
  const int split = 1 << a.split_log, share = ((dk + 15) / 16 + split - 1) / split * 16;
  const int col_boxes = (dv + 31) / 32;
  a.box_rows = std::min(col_boxes == 1 ? 128 : col_boxes == 2 ? 64 : 32, share);  // a stage, or a CTA's share
  a.heads = fast_div((uint32_t)c.H);
  a.per_qk = fast_div((uint32_t)(c.H / c.Hqk));
  const TreeLayout lay = tree_layout<T, NT>(dv, a.N, (int)c.levels);
  const size_t own_smem = (sizeof(TreeSmem) + 1023) & ~(size_t)1023;  // the stages begin at a multiple of 1024
  const size_t fixed = own_smem + 1024;                              // (1024 of each CTA are the system's)
  // as many CTAs on an SM as leave the ring three stages, one of them its own.  The last of its own holds the tree's decays
  // until the tokens are done with: where it is the only one (bf16: d_v from 96 on and 17 nodes or more), no page is on its
  // way before that
  const int later = lay.q / kStageBytes;
  int ctas = tree_ctas<T, NT>();
  while (ctas > 1 && fixed + lay.end + std::max(1, 3 - later) * kStageBytes > kSm / ctas) --ctas;
  a.own = (int)std::min<size_t>(kMaxTreeStages, (kSm / ctas - fixed - lay.end) / kStageBytes);
  if (ctas == 1) a.own = std::min(a.own, (int)((232448 - own_smem - lay.end) / kStageBytes));  // what a CTA can have
  a.stages = std::min(kMaxTreeStages, a.own + later);
  const size_t smem = (size_t)a.own * kStageBytes + lay.end;
  CUtensorMap pages;
  if (!make_pages_map(&pages, c.pages, c.n_pages, c.H, c.dk, c.dv, a.box_rows)) return cudaErrorInvalidValue;
  const auto kernel = cache_tree_kernel<T, NT>;
  const cudaError_t e = allow_shared(kernel);
  if (e != cudaSuccess) return e;
  return launch_following(false, kernel, dim3((unsigned)(items << a.split_log)), kTreeThreads, smem, split, s, pages, c, a);
}

// A tile for every 8 nodes, up to 64 of them; with fp32 tokens up to 32, whose two parts of everything are what
// shared memory and registers hold, and two groups above that.
template <typename T>
cudaError_t launch_nodes(const ll_cache& c, const TreeArgs& a, cudaStream_t s) {
  if (a.N <= 8) return launch<T, 1>(c, a, s);
  if (a.N <= 16) return launch<T, 2>(c, a, s);
  if (a.N <= 32 || sizeof(T) == 4) return launch<T, 4>(c, a, s);
  return launch<T, sizeof(T) == 4 ? 4 : 8>(c, a, s);
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
  return c.dtype == LL_F32 ? launch_nodes<float>(c, a, s) : launch_nodes<__nv_bfloat16>(c, a, s);
}

}  // namespace ll
