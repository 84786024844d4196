/*
 * loglinear.h — C ABI of the log-linear attention library (sm_103a).
 *
 * The operation (page "论文阅读：Log-Linear Attention — 基于 Fenwick 树与层次矩阵的对数线性
 * 复杂度注意力机制", sections 并行形式 and 与已有模型的组合; page "算力终结者来了！…", section
 * 结构矩阵):
 *
 *     O = (Q K^T ⊙ M^S ⊙ M^H) V,
 *     M^S[t,s] = prod_{r=s+1..t} a_r        (Mamba-2 scalar decay; all ones without it)
 *     M^H[t,s] = lambda[t, l(t,s)]           (Fenwick level l(t,s) of source s from query t)
 *
 * and its recurrent decode step with the lssb rule (first page, section 解码：基于 lssb 的
 * 状态更新).  l(t,t) = 0; for s < t, l(t,s) is the level of the Fenwick bucket of t holding s
 * (first page, section 层级判定算法), equal to the bit length of (t XOR s).
 *
 * Conventions shared by every entry point:
 *   - All tensor arguments are DEVICE pointers to dense row-major arrays, owned by the
 *     caller (loglinear_fwd_strided takes strided q, k, v and out).  The library never allocates, frees or synchronises; all work
 *     is enqueued on `stream` (NULL = the legacy default stream) and is asynchronous.
 *   - Sizes are element counts.  Positions t are 0-based and must fit in int32.
 *   - Every call validates its arguments on the host before launching anything and
 *     returns an ll_status code; on a non-zero status nothing has been enqueued, except
 *     LL_ERR_CUDA, which reports a failed launch (the message is in
 *     loglinear_last_cuda_error()).
 *   - `out` must not alias any input.  Calls are thread-safe.
 */
#ifndef LOGLINEAR_H
#define LOGLINEAR_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define LL_API __attribute__((visibility("default")))
#else
#define LL_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* ll_stream_t;

typedef enum {
  LL_OK = 0,
  LL_ERR_INVALID = 1,      /* a required pointer is NULL, a size is negative, unknown enum */
  LL_ERR_SHAPE = 2,        /* sizes violate the method: chunk not a power of two, too few levels */
  LL_ERR_DTYPE = 3,        /* unknown dtype code */
  LL_ERR_UNSUPPORTED = 4,  /* valid problem outside this build's kernels (e.g. head dim > 128) */
  LL_ERR_CUDA = 5,         /* a CUDA call or kernel launch failed */
  LL_ERR_WORKSPACE = 6,    /* workspace NULL or smaller than loglinear_fwd_workspace_size() */
  LL_ERR_ALIGN = 7         /* a pointer is not aligned as the chosen kernel path requires */
} ll_status;

typedef enum { LL_F32 = 0, LL_BF16 = 1 } ll_dtype;

/* Kernel path of the forward.  AUTO takes the tensor-core path when it applies (bf16
 * inputs, dk = 128, dv = 64 or 128) and the fp32 CUDA-core path otherwise. */
typedef enum { LL_PATH_AUTO = 0, LL_PATH_SIMT = 1, LL_PATH_TC = 2 } ll_path;

/* Library version, (major << 16) | minor. */
LL_API int loglinear_version(void);

/* Human-readable name of a status code (static string). */
LL_API const char* loglinear_status_string(int status);

/* Text of the last CUDA error seen by this thread (static per-thread buffer). */
LL_API const char* loglinear_last_cuda_error(void);

/* Path the forward would take for these arguments (LL_PATH_SIMT or LL_PATH_TC), or a
 * negative ll_status if the request is invalid. */
LL_API int loglinear_fwd_resolve_path(int64_t dk, int64_t dv, int chunk, int in_dtype, int path);

/*
 * Workspace bytes loglinear_fwd needs (written to *bytes).  The workspace holds the
 * per-chunk states U_i (chunk-local decayed sums of k v^T), the Fenwick block states the
 * inter-chunk readout uses, and the per-chunk log decays.  It is scratch: its content on
 * entry does not matter and is not meaningful on exit.
 */
LL_API int loglinear_fwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t dk, int64_t dv,
                                 int chunk, int in_dtype, int path, size_t* bytes);

/*
 * Chunked-parallel forward (first page, sections 矩阵分解 and 两阶段计算; second page,
 * section 高效训练算法): intra-chunk masked attention for the levels inside a chunk, per-
 * chunk states, a level scan over Fenwick block pairs of chunks, and a lambda-weighted
 * readout of the block states fused into the output epilogue.
 *
 *   q, k    [B, T, Hqk, dk] in_dtype (LL_F32 or LL_BF16).  Hqk q/k heads shared by the
 *                           H value heads in contiguous groups of H / Hqk: head h reads
 *                           q/k head h / (H / Hqk).  Hqk = H is one q/k per head; Hqk = 1
 *                           shares one q/k across all heads (Mamba-2's multi-value form).
 *                           1 <= Hqk <= H and H % Hqk == 0, else LL_ERR_SHAPE.
 *   v       [B, T, H, dv]   in_dtype
 *   log_a   [B, T, H]       fp32, log of the decay a_t (<= 0 expected); NULL = no decay
 *   lambda  [B, T, H, L]    fp32 level weights lambda[t, l]; L >= bit_length(T-1) + 1;
 *                           levels above bit_length(T-1) are not read
 *   out     [B, T, H, dv]   out_dtype (LL_F32 or LL_BF16), fully overwritten
 *   chunk   C, a power of two.  The result does not depend on C: the decomposition into
 *           an intra-chunk block D plus inter-chunk levels is exact for any C.  The fp32
 *           path works on chunks of min(C, 64) tokens; the tensor-core path on 128-token
 *           tiles (levels <= 7 in the dense intra-tile product, the rest through block
 *           states).
 *   T need not be a multiple of C (the last chunk is partial).  B, T or H = 0 is a no-op.
 *   workspace: device scratch of at least loglinear_fwd_workspace_size() bytes, 256-byte
 *           aligned.  Two calls that run concurrently need two workspaces.
 * Errors: LL_ERR_INVALID, LL_ERR_SHAPE, LL_ERR_DTYPE, LL_ERR_UNSUPPORTED (dk or dv > 128;
 * LL_PATH_TC forced on a shape other than bf16 with dk = 128, dv in {64, 128}), LL_ERR_WORKSPACE, LL_ERR_ALIGN (tensor-core
 * path: q, k, v, out not 16-byte aligned), LL_ERR_CUDA.
 */
LL_API int loglinear_fwd(const void* q, const void* k, const void* v, const float* log_a,
                  const float* lambda, void* out, int64_t B, int64_t T, int64_t H,
                  int64_t Hqk, int64_t dk, int64_t dv, int64_t L, int chunk, int in_dtype,
                  int out_dtype, int path, void* workspace, size_t workspace_bytes,
                  ll_stream_t stream);

/*
 * Element strides of a [B, T, Hx, width] tensor whose feature dimension (width) is
 * contiguous: the distance between consecutive batch entries, positions and heads.  A
 * dense tensor has {T*Hx*width, Hx*width, width}.  A q, k or v slice of a fused
 * [B, T, H, 3*d] projection has {T*H*3d, H*3d, 3d}.
 */
typedef struct {
  int64_t b, t, h;
} ll_strides;

/*
 * loglinear_fwd on strided q, k, v and out (each pointer addresses element [0, 0, 0, 0];
 * a NULL stride descriptor means dense).  log_a and lambda stay dense.  Same operation,
 * workspace and errors as loglinear_fwd, and in addition:
 *   LL_ERR_INVALID      a negative stride, or out strides under which two output
 *                       elements would share an address;
 *   LL_ERR_ALIGN        tensor-core path: a stride of a dimension longer than 1 that is not
 *                       a multiple of 16 bytes (8 bf16 or 4 fp32 elements), as TMA requires;
 *   LL_ERR_UNSUPPORTED  tensor-core path: a zero stride on a dimension longer than 1.
 * Strides of dimensions of size 1 are ignored.
 */
LL_API int loglinear_fwd_strided(const void* q, const ll_strides* q_strides, const void* k,
                                 const ll_strides* k_strides, const void* v,
                                 const ll_strides* v_strides, const float* log_a,
                                 const float* lambda, void* out, const ll_strides* out_strides,
                                 int64_t B, int64_t T, int64_t H, int64_t Hqk, int64_t dk,
                                 int64_t dv, int64_t L, int chunk, int in_dtype, int out_dtype,
                                 int path, void* workspace, size_t workspace_bytes,
                                 ll_stream_t stream);

/*
 * loglinear_fwd with per-kernel timing: identical work and results, plus cudaEventRecord
 * of stage_events[0] before the first kernel and of stage_events[i+1] after kernel i, on
 * `stream`.  stage_events is a host array of n_events cudaEvent_t handles created by the
 * caller; events past the number of kernels launched are recorded after the last one.
 * *n_kernels (if not NULL) receives the number of kernels launched.
 */
LL_API int loglinear_fwd_with_events(const void* q, const void* k, const void* v,
                                     const float* log_a, const float* lambda, void* out,
                                     int64_t B, int64_t T, int64_t H, int64_t Hqk, int64_t dk,
                                     int64_t dv,
                                     int64_t L, int chunk, int in_dtype, int out_dtype, int path,
                                     void* workspace, size_t workspace_bytes, ll_stream_t stream,
                                     void* const* stage_events, int n_events, int* n_kernels);

/*
 * Prefill for decoding: loglinear_fwd over positions 0..T-1, plus the per-level decode
 * state at position T-1, so that loglinear_decode_step can continue at t = T (first page,
 * sections 循环形式与输出计算 (one state per Fenwick bucket) and 两阶段计算 (block states
 * of chunks)).  Level l of the state is the sum over the level-l Fenwick bucket of T-1 of
 * exp(cum_{T-1} - cum_s) k_s v_s^T.  Levels above the last chunk are the forward's block
 * states of chunks, decayed to T-1; the levels inside the last chunk (and level 0) are
 * summed from k and v; the other levels are zero.
 *   state_out [B, H, L, dk, dv] fp32, fully overwritten (all zero when T = 0).  On the
 *           tensor-core path the levels taken from block states carry their bf16
 *           rounding.
 * The other arguments, the workspace and the errors are those of loglinear_fwd; state_out
 * NULL or not 4-byte aligned is LL_ERR_INVALID / LL_ERR_ALIGN.
 */
LL_API int loglinear_prefill(const void* q, const void* k, const void* v, const float* log_a,
                             const float* lambda, void* out, float* state_out, int64_t B,
                             int64_t T, int64_t H, int64_t Hqk, int64_t dk, int64_t dv,
                             int64_t L, int chunk,
                             int in_dtype, int out_dtype, int path, void* workspace,
                             size_t workspace_bytes, ll_stream_t stream);

/*
 * loglinear_prefill with per-kernel timing, as loglinear_fwd_with_events: stage_events[0]
 * is recorded before the first kernel and stage_events[i+1] after kernel i, the last of
 * which is the kernel that forms the decode state.  T = 0 launches no kernel and records
 * no event (*n_kernels = 0).
 */
LL_API int loglinear_prefill_with_events(const void* q, const void* k, const void* v,
                                         const float* log_a, const float* lambda, void* out,
                                         float* state_out, int64_t B, int64_t T, int64_t H,
                                         int64_t Hqk, int64_t dk, int64_t dv, int64_t L,
                                         int chunk, int in_dtype, int out_dtype, int path,
                                         void* workspace, size_t workspace_bytes,
                                         ll_stream_t stream, void* const* stage_events,
                                         int n_events, int* n_kernels);

/*
 * One decode step at position t for every (b, h) (first page, section 解码：基于 lssb 的
 * 状态更新; slide deck "論文紹介：Log Linear Attention", slide 21).  With l = lssb(t) (index of
 * the lowest set bit of t > 0):
 *   S^(l+1) <- a_t * sum_{j<=l} S^(j);  S^(1..l) <- 0;  S^(j) <- a_t * S^(j) for j > l+1;
 *   S^(0) <- k_t v_t^T;  out = sum_j lambda[j] * S^(j)^T q_t   (non-empty levels only).
 * At t = 0 the state is (re)initialised: S^(0) <- k_0 v_0^T, every other level <- 0.
 * For t > 0 the state must hold the Fenwick states after position t-1: the levels that
 * are empty after t-1 (bit j-1 of t-1 clear, j >= 1) are neither read nor written.
 *
 *   state   [B, H, L, dk, dv] fp32, updated in place, 16-byte aligned
 *   q, k    [B, Hqk, dk] in_dtype (q/k heads shared as in loglinear_fwd);
 *   v       [B, H, dv]   in_dtype
 *   log_a   [B, H] fp32 or NULL (no decay);   lambda [B, H, L] fp32
 *   out     [B, H, dv]   out_dtype, overwritten
 *   t       >= 0, same for every (b, h); L >= bit_length(t) + 1
 * Supported: 1 <= dk <= 128; dv a power of two in [4, 128].
 * Errors: LL_ERR_INVALID, LL_ERR_SHAPE, LL_ERR_DTYPE, LL_ERR_UNSUPPORTED, LL_ERR_ALIGN,
 * LL_ERR_CUDA.
 */
LL_API int loglinear_decode_step(float* state, const void* q, const void* k, const void* v,
                          const float* log_a, const float* lambda, int64_t t, void* out,
                          int64_t B, int64_t H, int64_t Hqk, int64_t dk, int64_t dv,
                          int64_t L, int in_dtype, int out_dtype, ll_stream_t stream);

/*
 * One decode step of Log-Linear Gated DeltaNet at position t for every (b, h).  The pages
 * build the log-linear form of a model by keeping its transition and composing its mask
 * with the Fenwick mask (page "算力终结者来了！…", section 对Mamba-2和门控DeltaNet的对数线性
 * 推广; first page, section 与已有模型的组合); the transition is the published gated delta
 * rule (Yang, Kautz and Hatamizadeh, "Gated Delta Networks", 2024).  With the state
 * stored [d_k][d_v] and A_t = alpha_t (I - beta_t k_t k_t^T), alpha_t = exp(log_a_t):
 *   every level that holds data after t-1:  S^(j) <- A_t S^(j);  then, with l = lssb(t),
 *   S^(l+1) <- sum_{j<=l} S^(j);  S^(1..l) <- 0;  S^(0) <- beta_t k_t v_t^T;
 *   out = sum_j lambda[j] * S^(j)^T q_t   (non-empty levels only).
 * At t = 0 the state is (re)initialised: S^(0) <- beta_0 k_0 v_0^T, every other level <- 0.
 * Lambda constant across levels gives plain Gated DeltaNet; without the k k^T term it is
 * loglinear_decode_step with v scaled by beta.
 *   state   [B, H, L, dk, dv] fp32, updated in place, 16-byte aligned (levels that are
 *           empty after t-1, other than lssb(t)+1, are neither read nor written)
 *   q, k    [B, Hqk, dk] in_dtype (q/k heads shared as in loglinear_fwd); k is expected
 *           to have unit length, as the gated delta rule assumes (not checked)
 *   v       [B, H, dv]   in_dtype
 *   log_a   [B, H] fp32 or NULL (alpha = 1);   beta [B, H] fp32;   lambda [B, H, L] fp32
 *   out     [B, H, dv]   out_dtype, overwritten
 *   t       >= 0, same for every (b, h); L >= bit_length(t) + 1
 * Supported: 1 <= dk <= 128; dv a power of two in [4, 128].
 * Errors: LL_ERR_INVALID (a NULL required pointer, beta included), LL_ERR_SHAPE,
 * LL_ERR_DTYPE, LL_ERR_UNSUPPORTED, LL_ERR_ALIGN, LL_ERR_CUDA.
 */
LL_API int loglinear_gdn_decode_step(float* state, const void* q, const void* k, const void* v,
                                     const float* log_a, const float* beta, const float* lambda,
                                     int64_t t, void* out, int64_t B, int64_t H, int64_t Hqk,
                                     int64_t dk, int64_t dv, int64_t L, int in_dtype,
                                     int out_dtype, ll_stream_t stream);

/*
 * Forward of Log-Linear Gated DeltaNet over a whole sequence, in the recurrent form: the
 * lssb step of loglinear_gdn_decode_step applied at t = 0..T-1 for every (b, h), with every
 * level's state kept on chip (same sources as loglinear_gdn_decode_step).  Equivalently
 *   o_t = sum_{s<=t} lambda[t, level(t, s)] beta_s (q_t^T A_t ... A_{s+1} k_s) v_s,
 * the model's own attention matrix composed with the Fenwick mask.
 *   q, k       [B, T, Hqk, dk] in_dtype, 4-byte aligned (heads shared as in loglinear_fwd);
 *              k is expected to have unit length (not checked)
 *   v          [B, T, H, dv] in_dtype
 *   log_a      [B, T, H] fp32 or NULL (alpha = 1);  beta [B, T, H] fp32
 *   lambda     [B, T, H, L] fp32, L >= bit_length(T-1) + 1
 *   out        [B, T, H, dv] out_dtype, overwritten
 *   state_out  NULL, or [B, H, L, dk, dv] fp32, overwritten with the per-level state after
 *              position T-1 (all zero for T = 0): the state loglinear_gdn_decode_step
 *              continues from at t = T
 * Supported: 1 <= dk, dv <= 128 (dk even for bf16), L <= 64.  The recurrence is sequential
 * in t (one CTA per (b, h, 8 columns of d_v)); the chunked form is not provided.
 * Errors: LL_ERR_INVALID, LL_ERR_SHAPE, LL_ERR_DTYPE, LL_ERR_UNSUPPORTED, LL_ERR_ALIGN,
 * LL_ERR_CUDA.
 */
LL_API int loglinear_gdn_fwd(const void* q, const void* k, const void* v, const float* log_a,
                             const float* beta, const float* lambda, void* out, float* state_out,
                             int64_t B, int64_t T, int64_t H, int64_t Hqk, int64_t dk, int64_t dv,
                             int64_t L, int in_dtype, int out_dtype, ll_stream_t stream);

/*
 * The same forward of Log-Linear Gated DeltaNet in chunks of 64 tokens, fp32 on CUDA cores:
 * per chunk the UT-transform form of the delta rule (Yang et al., "Parallelizing Linear
 * Transformers with the Delta Rule over Sequence Length", 2024) gives the chunk's own
 * attention matrix (masked by the Fenwick levels inside the chunk), its queries carried
 * back to the chunk start, its d_k x d_k transition and its own state; a sequential scan over
 * the chunks then carries every chunk-level block state by the chunk transitions, merges
 * them by the lssb rule on chunk indices and adds their lambda-weighted readout (first
 * page, sections 矩阵分解 and 两阶段计算, with the transition in place of the scalar decay).
 * Arguments as loglinear_gdn_fwd, plus a workspace of
 * loglinear_gdn_fwd_chunked_workspace_size() bytes (256-byte aligned; the chunks' partial
 * outputs, carried queries, transitions and states in fp32).  state_out (optional) receives
 * the decode state after T-1: the chunk-level states from the scan, the levels inside the
 * last chunk from the lssb steps over its tokens alone (then q and k must be 4-byte aligned
 * and, for bf16, dk even).  Otherwise no alignment is needed of q, k, v.  Supported:
 * 1 <= dk, dv <= 128, L <= 64, T <= 2^25.
 * Errors: LL_ERR_INVALID, LL_ERR_SHAPE, LL_ERR_DTYPE, LL_ERR_UNSUPPORTED, LL_ERR_WORKSPACE,
 * LL_ERR_ALIGN, LL_ERR_CUDA.
 */
LL_API int loglinear_gdn_fwd_chunked_workspace_size(int64_t B, int64_t T, int64_t H, int64_t dk,
                                                    int64_t dv, size_t* bytes);
LL_API int loglinear_gdn_fwd_chunked(const void* q, const void* k, const void* v,
                                     const float* log_a, const float* beta, const float* lambda,
                                     void* out, float* state_out, int64_t B, int64_t T,
                                     int64_t H, int64_t Hqk,
                                     int64_t dk, int64_t dv, int64_t L, int in_dtype,
                                     int out_dtype, void* workspace, size_t workspace_bytes,
                                     ll_stream_t stream);

/*
 * Backward of loglinear_fwd (page "算力终结者来了！…", sections 结构矩阵 and 讨论与局限性:
 * training takes the gradients of the attention terms and of the level weights lambda):
 * given dout = dL/dO, the gradients of L with respect to every input, for
 * O = (Q K^T ⊙ M^S ⊙ M^H) V exactly as loglinear_fwd defines it:
 *   dq, dk  [B, T, Hqk, dk]  grad_dtype (summed over the heads that share a q/k head)
 *   dv      [B, T, H, dv]    grad_dtype
 *   dlog_a  [B, T, H] fp32   (required when log_a is given; ignored when log_a is NULL)
 *   dlambda [B, T, H, L] fp32 (levels above bit_length(T-1) receive 0)
 *   dout    [B, T, H, dv]    grad_dtype
 * q, k, v, log_a, lambda, B, T, H, Hqk, dk, dv and L as in loglinear_fwd; no chunk
 * argument: the gradients do not depend on it.  1 <= dk, dv <= 128, L <= 64.  All
 * outputs are fully overwritten.
 * path: LL_PATH_TC computes dq, dk, dv and dlambda on the tensor cores (bf16 inputs and
 *   gradients, dk = 128, dv in {64, 128}; q, k, v, dout, dq, dk, dv 16-byte aligned): the
 *   tensor-core forward, in a form that writes no output, publishes its block states into
 *   the workspace; 128-token tiles take dQ and dlambda from them with tcgen05; the
 *   mirrored states of later tiles that dk and dv read are summed per Fenwick slot with
 *   tcgen05 (fp32 accumulation, the scaled q split into a bf16 high part and residual),
 *   then dK and dV are formed per 128-token tile with tcgen05.  These carry the bf16
 *   roundings of P, P' and of the states.  LL_PATH_SIMT computes everything on CUDA cores
 *   in fp32.
 *   LL_PATH_AUTO takes the tensor cores when they apply.  The workspace size depends on
 *   the path.
 * fwd_workspace: NULL, or, on the tensor-core path, the workspace of a loglinear_fwd call
 *   that ran on the tensor-core path (LL_PATH_TC or AUTO with bf16, dk = 128) over these
 *   same q, k, v, log_a, lambda and sizes, with nothing written to it since.  Its block
 *   states are then read instead of being recomputed by a forward inside this call (the
 *   usual training step: forward, then backward).  The library cannot check that the
 *   contents match the inputs; that is the caller's contract.  It does check, on the GPU,
 *   the layout tag the tensor-core forward leaves in its workspace (sizes and path): a
 *   mismatch raises bit 2 of loglinear_device_error.  fwd_workspace_bytes must
 *   be at least loglinear_fwd_workspace_size() for the forward's arguments
 *   (LL_ERR_WORKSPACE); a non-NULL fwd_workspace on the CUDA-core path is
 *   LL_ERR_UNSUPPORTED.  An empty call (B, T or H zero) returns LL_OK before any of
 *   these checks of pointers and workspaces.
 * workspace: device scratch of at least loglinear_bwd_workspace_size() bytes, 256-byte
 * aligned (recomputed forward states, per-head q and k gradients).
 * Errors: LL_ERR_INVALID (null pointer, negative size, dlog_a NULL with log_a given),
 * LL_ERR_SHAPE (L too small, Hqk not dividing H), LL_ERR_DTYPE, LL_ERR_UNSUPPORTED,
 * LL_ERR_WORKSPACE, LL_ERR_ALIGN (workspace), LL_ERR_CUDA.
 */
LL_API int loglinear_bwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t Hqk,
                                        int64_t dk, int64_t dv, int64_t L, int in_dtype,
                                        int grad_dtype, int path, size_t* bytes);
LL_API int loglinear_bwd(const void* q, const void* k, const void* v, const float* log_a,
                         const float* lambda, const void* dout, void* dq, void* dk, void* dv,
                         float* dlog_a, float* dlambda, int64_t B, int64_t T, int64_t H,
                         int64_t Hqk, int64_t dk_dim, int64_t dv_dim, int64_t L, int in_dtype,
                         int grad_dtype, int path, const void* fwd_workspace,
                         size_t fwd_workspace_bytes, void* workspace, size_t workspace_bytes,
                         ll_stream_t stream);

/*
 * Reads and clears the device error word of the tensor-core path (synchronises `stream`).
 * *flags = 0 when every wait of the kernels run so far completed.  Bit 0: an mbarrier
 * wait ran out of time (the CTA then skipped its remaining work and its output tile is
 * not valid).  Bit 1: a wait for another tile's published state ran out of time (the
 * output of that tile is not valid).  Bit 2: loglinear_bwd was given a fwd_workspace
 * that a tensor-core loglinear_fwd with the same B, T, H, Hqk and dv did not write (its
 * layout tag does not match; the gradients are not valid).  Bit 3: a wait inside loglinear_glr_fwd or
 * _bwd ran out of time (the results are not valid).  Bit 4: loglinear_glr_step was given a
 * slot out of range, or one that an earlier row has (that row was left out).  Bit 5:
 * loglinear_tree_verify was given a row that is no tree, or a token outside the vocabulary (that
 * row accepted nothing).  The launch itself still reported success.
 */
LL_API int loglinear_device_error(ll_stream_t stream, unsigned* flags);

/*
 * Gated linear recurrence, per channel:
 *     h_t = a_t h_{t-1} + b_t x_t,   a_t = exp(log_a_t),
 *     b_t = 1 (LL_GLR_NONE), 1 - a_t (LL_GLR_ONE_MINUS) or sqrt(1 - a_t^2) (LL_GLR_SQRT).
 * The vector-state recurrence of gated layers that stand between attention layers; the
 * sources have no counterpart.  One pass: every input is read once, every output written once.
 *   x          [B, T, D] in_dtype; log_a [B, T, D] gate_dtype (<= 0 expected; -inf is a = 0).
 *              gate_dtype is LL_F32 or in_dtype (else LL_ERR_UNSUPPORTED).  Both may be
 *              strided: element strides of the batch and position dimensions (h is not
 *              read), channels contiguous; NULL = dense.
 *   cu_seqlens NULL: B sequences of T tokens.  Else device int32 [N + 1], 0 = cu[0] <= cu[1]
 *              <= ... <= T, with B = 1: sequence n holds tokens cu[n] .. cu[n+1] - 1, and
 *              nothing passes from one to the next, infinities and NaN included.  Rows
 *              behind cu[N] may hold anything, and their outputs (and gradients) are left as
 *              they were.  The library does not read the bounds
 *              on the host; bounds out of order give wrong sequences, but no access outside
 *              the arrays.
 *   N          number of sequences (ignored without cu_seqlens: B)
 *   h0         [N, D] fp32 state before the first token; NULL = zero
 *   out        [B, T, D] out_dtype: h_t
 *   state_out  NULL, or [N, D] fp32: the state after the last token (h0 for an empty sequence);
 *              may be h0 itself
 * State, gates and sums are fp32; out is rounded once.  Gates below 2^-126 are 0.  An infinite state
 * stays infinite through gates that are not 0, however many, and is NaN behind one that is, as
 * token by token; but runs of tokens are summed before the state that comes into them is added, so
 * what only passes fp32's range in between may do so in one order and not in the other.
 * Errors: LL_ERR_INVALID (null pointer, negative size or stride, unknown scale, cu_seqlens with
 * B other than 1), LL_ERR_DTYPE, LL_ERR_UNSUPPORTED (T or N > 2^30, B or D or B * ceil(D / 32) above
 * 2^27), LL_ERR_ALIGN (a pointer not aligned to its element), LL_ERR_CUDA.  B, T or D = 0 is a no-op, but that state_out still receives h0.
 */
typedef enum { LL_GLR_NONE = 0, LL_GLR_ONE_MINUS = 1, LL_GLR_SQRT = 2 } ll_glr_scale;

LL_API int loglinear_glr_fwd(const void* x, const ll_strides* x_strides, const void* log_a,
                             const ll_strides* log_a_strides, const float* h0,
                             const int32_t* cu_seqlens, int64_t N, void* out, float* state_out,
                             int64_t B, int64_t T, int64_t D, int in_dtype, int gate_dtype,
                             int out_dtype, int scale, ll_stream_t stream);

/*
 * Gradients of loglinear_glr_fwd, given dout = dL/d out and (or NULL) dstate = dL/d state_out:
 *     g_t = dout_t + a_{t+1} g_{t+1}  (+ dstate at the sequence's last token)
 *     dx_t = b_t g_t,   dlog_a_t = a_t h_{t-1} g_t + b'(log_a_t) x_t g_t,   dh0 = a g at the first
 * h is the forward's out (its rounding enters dlog_a).  Where b = sqrt(1 - a^2) is 0, its
 * derivative, which is infinite, is taken as 0.
 *   h, dout, dx   [B, T, D] grad_dtype, dense;  dlog_a [B, T, D] gate_dtype, dense
 *   x             may be NULL with LL_GLR_NONE, whose gradients do not read it
 *   dstate, dh0   [N, D] fp32 or NULL (dh0 of an empty sequence is its dstate, or zero); may be
 *                 the same array
 * x, log_a, h0, cu_seqlens, N, sizes and errors as loglinear_glr_fwd.
 */
LL_API int loglinear_glr_bwd(const void* x, const ll_strides* x_strides, const void* log_a,
                             const ll_strides* log_a_strides, const float* h0,
                             const int32_t* cu_seqlens, int64_t N, const void* h,
                             const void* dout, const float* dstate, void* dx, void* dlog_a,
                             float* dh0, int64_t B, int64_t T, int64_t D, int in_dtype,
                             int gate_dtype, int grad_dtype, int scale, ll_stream_t stream);

/*
 * One token of the recurrence for each of B rows: state[slot] <- a state[slot] + b x, out = the new
 * state.
 *   state  [S, D] fp32, updated in place;  x [B, D] in_dtype;  log_a [B, D] gate_dtype
 *   slots  NULL (row b has slot b; then S >= B, else LL_ERR_SHAPE), or device int32 [B]: the
 *          row's slot; -1 leaves the row out (its out is not written).  A slot out of range, or
 *          one that an earlier row has, leaves the row out too and raises bit 4 of
 *          loglinear_device_error.
 *   out    [B, D] out_dtype
 * Errors: LL_ERR_INVALID, LL_ERR_SHAPE, LL_ERR_DTYPE, LL_ERR_UNSUPPORTED (B > 65535),
 * LL_ERR_ALIGN, LL_ERR_CUDA.
 */
LL_API int loglinear_glr_step(float* state, int64_t S, const int32_t* slots, const void* x,
                              const void* log_a, void* out, int64_t B, int64_t D, int in_dtype,
                              int gate_dtype, int out_dtype, int scale, ll_stream_t stream);

/*
 * The paged decode cache: decoding for sequences that are each at a position of their own.
 *
 * loglinear_decode_step keeps a dense state [B, H, L, dk, dv] whose rows are all at one
 * position, and reads and rewrites every level that holds data.  The cache keeps, for a slot
 * that holds n positions, the raw tokens of its current block (n mod 64 of them; the levels
 * inside a block are summed from them), and for every set bit i of j = n / 64 one page
 * [H, dk, dv] fp32: the state of the aligned run of 2^i blocks that the Fenwick partition has
 * there (token level 7 + i), as it was at its last token.  Its decay since then is one
 * number per head.  Pages are written once, at a block's last token, and may be shared.
 *
 * Every array is the caller's.  `free` below: a page with reference count 0; the lowest free
 * pages are taken first, in the order of the rows.  A new cache has page_table all -1 and
 * refcount all 0; the other arrays need no initial value.
 */
#define LL_CACHE_BLOCK 64

typedef struct {
  int64_t slots, n_pages;  /* >= 1; n_pages <= 2^30 */
  int64_t H, Hqk, dk, dv;  /* Hqk divides H; 1 <= dk <= 128; dv a multiple of 4, 4 <= dv <= 128 */
  int64_t levels;          /* M: pages a slot can hold, 1 <= M <= 24; a slot holds fewer than
                              64 * 2^M positions */
  int dtype;               /* LL_F32 or LL_BF16: the type of k and v */
  float* pages;            /* [n_pages, H, dk, dv], 16-byte aligned */
  int32_t* page_table;     /* [slots, M]: the page of each level, or -1 */
  int32_t* refcount;       /* [n_pages]: slots that hold the page */
  void* win_k;             /* [slots, Hqk, 64, dk] dtype: the block's keys; 16-byte aligned */
  void* win_v;             /* [slots, H, 64, dv] dtype: its values; 16-byte aligned */
  float* win_log_a;        /* [slots, H, 64]: its log decays */
  float* page_log;         /* [slots, 2, M, H]: for blocks of even and of odd number, each page's
                              log decay from its last token to the block's start */
  int32_t* page_from;      /* [slots, 2]: token of the block from which pages decay on */
  int32_t* scratch;        /* loglinear_cache_scratch_size() bytes */
  uint32_t* error;         /* [1] bits below, raised by kernels; the caller reads and clears it */
} ll_cache;

/* Raised on the device by rows that are then left out (their slot and output as they were). */
#define LL_CACHE_ERR_SLOT 1u      /* slot out of range (other than -1), or given to an earlier row */
#define LL_CACHE_ERR_POSITION 2u  /* position outside the cache, or before the end of the prompt that
                                     was loaded, in a block with pages */
#define LL_CACHE_ERR_PAGES 4u     /* no free page was left (the slot is left without it) */
#define LL_CACHE_ERR_MISSING 8u   /* a page that the position needs is not there, or the page that
                                     a step would fold into is shared (not reserved) */
#define LL_CACHE_ERR_WAIT 16u     /* a wait inside loglinear_cache_step or _tree ran out of time; the rows'
                                     results are not valid */
#define LL_CACHE_ERR_TREE 32u     /* a node's parent does not come before it or is left out, or a path
                                     names a node that is not there */

LL_API int loglinear_cache_scratch_size(int64_t slots, int64_t n_pages, size_t* bytes);

/*
 * Conventions of the calls on a cache: `slots` (and src, dst) device int32 [n], -1 leaves the row
 * out; `pos` device int32 [n], the positions each row's slot holds, read from device memory so
 * that a captured graph can be replayed.  Calls on one cache have to be ordered (one stream, or
 * events); its arrays are read and written by all of them.  n = 0 is a no-op.
 * Errors: LL_ERR_INVALID (null pointer or descriptor, negative size), LL_ERR_SHAPE (Hqk, too few
 * levels L), LL_ERR_DTYPE, LL_ERR_UNSUPPORTED (sizes outside the descriptor's limits, too many
 * rows for a launch), LL_ERR_ALIGN, LL_ERR_CUDA.
 */

/*
 * The page reservation that goes before a step at the same positions: each slot gives up the
 * pages that are no longer live at pos and, where pos is a block's last position, takes the
 * page that the block is folded into.  Needed at a block's last position; at other positions it
 * only gives pages back to the pool (at a block's first one).  May be repeated.
 */
LL_API int loglinear_cache_reserve(const ll_cache* cache, const int32_t* slots,
                                   const int32_t* pos, int64_t n, ll_stream_t stream);

/*
 * One decode step for n rows, each at its own position t = pos[row] (the definition of
 * loglinear_decode_step):
 *     out = sum_{s <= t} lambda[level(t, s)] exp(sum_{u=s+1..t} log_a_u) (q_t . k_s) v_s,
 * with the sum over whole blocks taken from the pages.  The token joins the slot's block; at a
 * block's last position the pages below level ctz(j + 1) and the block are folded into the page
 * of that level.  Repeating a step at the same position repeats its result, and a slot may go back
 * to earlier positions of the block (rejected drafts), its end included; but only until a call has
 * been made for it at a position of the next block, whose tokens replace the block's and whose
 * reservation gives up its pages, and not to before the end of a loaded prompt where the block
 * has pages.  Drafts that cross a block's end belong on a fork, or go through loglinear_cache_tree and
 * loglinear_cache_accept.
 *   q, k   [n, Hqk, dk] cache dtype;  v [n, H, dv] cache dtype
 *   log_a  [n, H] fp32 or NULL (no decay);  lambda [n, H, L] fp32, L >= M + 7
 *   out    [n, H, dv] out_dtype
 * pos below 64 * 2^M - 1.
 */
LL_API int loglinear_cache_step(const ll_cache* cache, const int32_t* slots, const int32_t* pos,
                                const void* q, const void* k, const void* v, const float* log_a,
                                const float* lambda, void* out, int64_t n, int64_t L,
                                int out_dtype, ll_stream_t stream);

/*
 * Puts n prompts of T positions into their slots, which give up what they held: the dense
 * states after position T - 1 as loglinear_prefill writes them, and the last T mod 64 tokens.
 * Where T is a multiple of 64 the levels that a step at T would merge are added into one page.
 *   state     [n, H, L, dk, dv] fp32, 16-byte aligned; L >= bit_length(T - 1) + 1
 *   k, v      the prompt's last Tk tokens, [n, Tk, Hqk, dk] and [n, Tk, H, dv] cache dtype,
 *             Tk >= T mod 64;  log_a [n, Tk, H] fp32 or NULL.  Element strides of the batch,
 *             position and head dimensions (features contiguous); NULL = dense.
 */
LL_API int loglinear_cache_load(const ll_cache* cache, const int32_t* slots, int64_t n,
                                int64_t T, const float* state, int64_t L, const void* k,
                                const ll_strides* k_strides, const void* v,
                                const ll_strides* v_strides, const float* log_a,
                                const ll_strides* log_a_strides, int64_t Tk, ll_stream_t stream);

/*
 * Dense states of n slots that hold pos[row] positions, from which loglinear_decode_step goes on
 * at t = pos[row] (or loglinear_cache_load on another cache).  Levels that are empty are zero.
 * Where pos is a multiple of 64, the levels that step pos merges are given as their sum, in
 * the highest of them, lssb(pos).  A slot may be given twice.
 *   state_out [n, H, L, dk, dv] fp32, 16-byte aligned; L >= M + 7
 */
LL_API int loglinear_cache_store(const ll_cache* cache, const int32_t* slots, const int32_t* pos,
                                 float* state_out, int64_t n, int64_t L, ll_stream_t stream);

/*
 * Slot dst[row] becomes a copy of slot src[row], which holds pos[row] positions; what it held is
 * given up.  Pages are shared, the block's tokens copied.  A source may be given many times; a
 * target is given once and is no row's source.
 */
LL_API int loglinear_cache_fork(const ll_cache* cache, const int32_t* src, const int32_t* dst,
                                const int32_t* pos, int64_t n, ll_stream_t stream);

/* The slots give up their pages. */
LL_API int loglinear_cache_free(const ll_cache* cache, const int32_t* slots, int64_t n,
                                ll_stream_t stream);

/*
 * Moves pages so that those in use are the lowest: the i-th lowest free page below their number
 * takes the i-th lowest page in use above it.  *n_live (device int32) receives their number;
 * the pages from there on are free.
 */
LL_API int loglinear_cache_compact(const ll_cache* cache, int32_t* n_live, ll_stream_t stream);

/*
 * Speculative decoding over the cache.  A round takes, per sequence, a tree of N drafted tokens
 * whose node 0 is the pending token (sampled last, not yet in the cache): loglinear_cache_tree
 * runs the layers' attention for all nodes, loglinear_tree_verify settles which drafts stand and draws
 * the next pending token, and loglinear_cache_accept puts the accepted path into the cache.
 *
 * parents: device int32 [n, N], 1 <= N <= LL_TREE_MAX.  A node's parent comes before it; -1: it
 * has none (depth 0: it follows the context); -2: the node is left out (padding), and so has no
 * children.  A parent that is not before its node, below -2, or left out is an error of the row.
 */
#define LL_TREE_MAX 64

/*
 * The decode step's attention for the nodes of a tree behind each slot's pos[row] positions, of
 * which nothing is written: node i at depth d stands at t = pos[row] + d, and
 *     out_i = sum_s lambda_i[level(t, s)] exp(sum of log_a behind s up to t) (q_i . k_s) v_s
 * over the context, the nodes above it and itself.  A tree may run over the end of a block, with no
 * fork or reservation; a slot may be given by many rows.  A node's output depends on its own
 * path alone, infinities and NaN in other nodes included.
 *   parents [n, N];  q, k [n, N, Hqk, dk], v [n, N, H, dv] cache dtype, strided as in
 *           loglinear_cache_load (batch, node, head; NULL = dense)
 *   log_a   [n, N, H] fp32 or NULL (no decay);  lambda [n, N, H, L] fp32, L >= M + 7
 *   out     [n, N, H, dv] out_dtype; rows with slot -1 and nodes that are left out are not written
 * Every node's t below 64 * 2^M - 1 (else POSITION).  A row that cannot be served is left out and
 * raises the cache's error word.  Errors as the cache's calls; LL_ERR_UNSUPPORTED: N > LL_TREE_MAX;
 * LL_ERR_INVALID: N < 1, a negative stride.
 */
LL_API int loglinear_cache_tree(const ll_cache* cache, const int32_t* slots, const int32_t* pos,
                                const int32_t* parents, const void* q, const ll_strides* q_strides,
                                const void* k, const ll_strides* k_strides, const void* v,
                                const ll_strides* v_strides, const float* log_a,
                                const float* lambda, void* out, int64_t n, int64_t N, int64_t L,
                                int out_dtype, ll_stream_t stream);

/*
 * The nodes path[row][0], path[row][1], ... (up to the first -1) join the slot at pos[row],
 * pos[row] + 1, ..., as steps there would have left them: tokens, and at a block's end the fold.
 * The reservation is included: the slot gives up pages that are no longer live at pos and, where
 * the path ends the block, takes the page of the fold, lowest free pages first, in the order of the
 * rows.  May be repeated at the same position (other drafts), unless the path went into the next
 * block, whose tokens replace the block's.
 *   path    device int32 [n, D], 1 <= D <= LL_TREE_MAX: nodes, in [0, N); whether they are a
 *           path of the tree is not checked.  Empty (-1 first): only the reservation
 *   k, v, log_a  the tree's, as in loglinear_cache_tree
 *   new_pos device int32 [n], not pos itself: pos[row] + the path's length; rows that are left out
 *           keep theirs
 * A slot given to an earlier row, a path that is too long for the cache, names no node, or folds
 * without its pages: the row is left out (in the last case with what it could reserve) and the error
 * word raised.
 */
LL_API int loglinear_cache_accept(const ll_cache* cache, const int32_t* slots, const int32_t* pos,
                                  const int32_t* path, const void* k, const ll_strides* k_strides,
                                  const void* v, const ll_strides* v_strides, const float* log_a,
                                  int32_t* new_pos, int64_t n, int64_t N, int64_t D,
                                  ll_stream_t stream);

/*
 * Verification of drafts by speculative sampling: where the rows of probs (and of draft) sum to 1, the
 * accepted tokens and the next one are distributed as the target's.  (Z starts at 1, not at the row's
 * own sum: a sum that is off by e moves a draft's chance by about e; rounded to bf16, up to 2^-8.)
 * The walk starts at node 0 and tries the current node's children in the order of their index, with
 * R the target's row P of that node and Z = 1 at first.  Node i, token x:
 *     draft NULL (drafts that were given, such as the likeliest tokens): accepted where u_i Z < R(x);
 *         else R(x) is taken off Z and set to 0.
 *     draft (each child drawn from its parent's row Q of it, independently): accepted where
 *         u_i Z Q(x) < R(x); else R <- max(R - Z Q, 0) and Z <- the sum of R.
 * Where none is accepted, the next token is the lowest index at which the running sum of R is above
 * u_0 times its whole (of P, where R is all 0; -1, where P is too).
 *   parents, tokens  int32 [n, N];  tokens of nodes with a parent in [0, V)
 *   probs, draft     [n, N, V] dtype (LL_F32 or LL_BF16): the distribution of the token after each node
 *                    by the target and (or NULL) by the model that drafted; values outside [0, 1] count
 *                    as the nearer bound, NaN as 0.  Rows of nodes that the walk does not reach are not
 *                    read, but for their children's tokens' values
 *   u                [n, N] fp32 in [0, 1) (others count as the nearest, NaN as 0); u_0 draws the token
 *   path             [n, N] int32: node 0, the accepted nodes, then -1;  count [n] int32: their number
 *   token            [n] int32: the next pending token
 * A row whose node 0 is left out (-2) gets an empty path and token -1.  One that is no tree, whose
 * node 0 is no root or that has a token outside the vocabulary does too, and raises bit 5 of
 * loglinear_device_error.  Sums are exact, of values rounded to the nearest 2^-43, and the same in any
 * order: the results do not depend on the launch.  (Rows whose values sum to 2^18 or more overflow: the
 * token is then any in the vocabulary, or -1.  With draft, the sum of the rejections' Z at one node
 * counts as at most 2^19, which matters where rows sum to more than 2^13: R can then be too large at
 * tokens whose Q is below 2^-19.)
 * Errors: LL_ERR_INVALID (null pointer, negative size, N or V < 1), LL_ERR_DTYPE,
 * LL_ERR_UNSUPPORTED (N > LL_TREE_MAX, V > 2^30, n > 2^24), LL_ERR_ALIGN, LL_ERR_CUDA.  n = 0 is a no-op.
 */
LL_API int loglinear_tree_verify(const int32_t* parents, const int32_t* tokens, const void* probs,
                                 const void* draft, const float* u, int32_t* path, int32_t* count,
                                 int32_t* token, int64_t n, int64_t N, int64_t V, int dtype,
                                 ll_stream_t stream);

/*
 * loglinear_fwd for callers that cannot allocate device memory.  The paper has no
 * counterpart to this entry point: it exists for callers such as a plugin inside a host
 * application that owns all device memory and hands extensions no allocator, or a
 * real-time loop where cudaMalloc (which may synchronise the device) is not allowed.
 *
 * Same arguments and result as loglinear_fwd, minus the workspace.  The scratch lives in
 * one fixed device array of LL_FWD_NOALLOC_SCRATCH_BYTES that the library declares; every
 * GPU that loads the library's device code holds it until the process exits.  This call
 * allocates nothing (no cudaMalloc, no allocating library routine).
 *   - The first call on a device (with that device current) looks up the array's device
 *     address and caches it with the ID of the current CUDA context; make that first call
 *     before any stream capture.  A call under a different context (after
 *     cudaDeviceReset, or when the application replaced the primary context) looks the
 *     address up again; make it, too, outside any stream capture.
 *   - The ready flags and the tile counter in the array are zeroed by every call, on
 *     `stream`, before the kernel that reads them; everything else in it is written
 *     before it is read.
 *   - All calls share the array and it keeps the last call's contents.  Nothing in it
 *     needs clearing between calls, but calls whose work overlaps on the GPU (another
 *     stream, another host thread) race on it: serialise them.
 *   - A problem whose scratch (loglinear_fwd_workspace_size) exceeds the array is
 *     rejected with LL_ERR_WORKSPACE before any launch.
 * Errors: those of loglinear_fwd; LL_ERR_WORKSPACE for problems too large; LL_ERR_CUDA if
 * the array's address cannot be obtained.
 */
#define LL_FWD_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
LL_API int loglinear_fwd_noalloc(const void* q, const void* k, const void* v,
                                 const float* log_a, const float* lambda, void* out,
                                 int64_t B, int64_t T, int64_t H, int64_t Hqk, int64_t dk,
                                 int64_t dv, int64_t L, int chunk, int in_dtype, int out_dtype,
                                 int path, ll_stream_t stream);

/*
 * Debug view of the forward's level indexing (first page, sections 层级判定算法 and 矩阵
 * 分解): writes levels[t * T + s] (int8, device) for 0 <= s, t < T: the Fenwick level the
 * given path assigns to the pair (query t, source s) through its intra-chunk formula or
 * its inter-chunk block pairing, and -1 for s > t.  chunk and path as in loglinear_fwd
 * (path AUTO resolves as for bf16, dk = dv = 128; the level map does not depend on dv).  T <= 16384.
 */
LL_API int loglinear_debug_level_map(int64_t T, int chunk, int path, int8_t* levels,
                              ll_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LOGLINEAR_H */
