/*
 * moe_decode.h — C ABI of the GB300 (sm_103a) MoE decode-layer library.
 *
 * The library computes the memory-bound decode step of a large MoE
 * transformer at batch M = 1..64 on one GPU: weight-streaming projections
 * chosen by batch size, the out-projection fused with its residual, sigmoid
 * router scoring with top-k, and the routed and shared SwiGLU experts.
 * Sources (the vLLM "Kimi K3" decode article and its summaries):
 *   [K3 P1§1] Part 1 §1 "Ajustar las formas": small-matrix kernels at batch
 *             1-2, split-K kernels at larger batch, for the projections.
 *   [K3 P1§2] Part 1 §2 "Superposición de computación y comunicación": the
 *             attention out-projection fused with the residual after it.
 *   [K3 P1§3] Part 1 §3 "Mejorar la programación de MoE": router scores,
 *             routed experts, the shared expert on a separate stream.
 *   [K3 P1§4] Part 1 §4 "Prefetching": small-batch decode is bound by weight
 *             reads; a side-stream kernel warms the cache with the next
 *             operator's weights during phases that leave bandwidth idle.
 *   [hu-sum]  aihirek.info summary, "Kevesebb kernel, összehangoltabb
 *             végrehajtás": the same kernel choice by batch size.
 *
 * Conventions (all entry points):
 *  - Tensors are caller-owned DEVICE memory, row-major. Weights use the
 *    nn.Linear layout W[N][K] (K contiguous), so y = x W^T. bf16 values are
 *    passed as their 16-bit patterns (dec_bf16). Every pointer must be
 *    16-byte aligned and every K (inner extent) a multiple of 8.
 *  - Calls are asynchronous on the given stream and never allocate device
 *    memory. Scratch space is the caller's workspace `ws` of `ws_bytes`
 *    bytes, sized by the matching *_workspace_size() query. A workspace must
 *    be zeroed (dec_workspace_init) before its first use and before it is
 *    reused by a call of another entry point or another shape; calls of the
 *    same entry point and shape leave it ready for the next one. One
 *    workspace must not be used by two calls that can run at the same time.
 *  - Arguments are checked on the host before anything is launched; a bad
 *    argument returns DEC_ERR_INVALID_ARG or DEC_ERR_UNSUPPORTED and launches
 *    nothing. A failed launch returns DEC_ERR_CUDA. No call aborts, exits or
 *    traps. Device waits are bounded: a wait that runs past the handle's
 *    limit makes its kernel stop early and sets the handle's device error
 *    word, which dec_check_device_error() reports as DEC_ERR_TIMEOUT.
 *  - Accumulation is fp32 everywhere; each bf16 output is rounded once.
 *  - A handle serves one thread at a time (it holds the side streams,
 *    events and the last-variant record).
 */
#ifndef MOE_DECODE_H
#define MOE_DECODE_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t dec_bf16; /* bit pattern of a bfloat16 value */

typedef enum dec_status {
  DEC_OK = 0,
  DEC_ERR_INVALID_ARG = 1, /* null or misaligned pointer, size out of range, workspace too small */
  DEC_ERR_UNSUPPORTED = 2, /* well-formed request outside the implemented shapes */
  DEC_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed */
  DEC_ERR_TIMEOUT = 4      /* a device wait ran past its limit (see dec_check_device_error) */
} dec_status;

/* Kernel families of the projections [K3 P1§1]. */
typedef enum dec_variant {
  DEC_VARIANT_AUTO = 0,    /* choose by batch and size (measured on GB300): SMALL_M for M <= 2, and for
                              M <= 4 when the weight matrix is at most 48 MB; SPLIT_K otherwise */
  DEC_VARIANT_SMALL_M = 1, /* CUDA-core small-matrix kernel: each CTA streams whole weight rows */
  DEC_VARIANT_SPLIT_K = 2  /* tcgen05 kernel; the weight k-blocks are split evenly over all SMs */
} dec_variant;

typedef struct dec_handle dec_handle;

/* ------------------------------------------------------------------ handle */

/* Create a handle on CUDA device `device`. The handle owns two side streams
 * (shared expert, L2 prefetch), their fork/join events and a 4-byte device
 * error word; nothing else. Returns DEC_ERR_CUDA if the device is absent. */
dec_status dec_create(dec_handle** out, int device);

/* Destroy a handle (synchronises its side streams first). NULL is allowed. */
dec_status dec_destroy(dec_handle* h);

/* Static description of a status code. Never NULL. */
const char* dec_status_string(dec_status s);

/* Zero a workspace before its first use (cudaMemsetAsync on `stream`). */
dec_status dec_workspace_init(dec_handle* h, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Limit, in nanoseconds, of every device-side wait (default 500 ms). */
dec_status dec_set_wait_limit_ns(dec_handle* h, uint64_t ns);

/* Enable (1, default) or disable (0) programmatic dependent launch: kernels
 * start while their predecessor drains and stream static weights before
 * waiting for it [K3 Part 2, "Validar la corrección": activation reads stay
 * behind the dependency wait, weight reads may go before it]. */
dec_status dec_set_pdl(dec_handle* h, int enable);

/* How the shared expert and the routed experts share the SMs [K3 P1§3: the
 * schedule sets how many GPU resources each operation uses]. The shared
 * expert is always launched first, beside the router / top-k phase.
 *  0 (default): it keeps its share of the expected weight bytes (rounded
 *     up), except from four tokens on with a shared expert of at least 48 MB,
 *     where it acts as -1 (measured on GB300: as fast with independent
 *     tokens, up to 17% faster when tokens share experts, as the drafts of a
 *     speculative-verify batch do; with a small shared expert the byte share
 *     is faster);
 * -1: it starts on every SM and the routed experts take SMs as it finishes;
 *  n > 0: it keeps n SMs. */
dec_status dec_set_shared_sms(dec_handle* h, int sms);

/* The small-matrix kernels (batch 1) keep about `bytes` of each CTA's
 * upcoming weight rows requested into L2 (bulk L2 prefetches, issued from
 * before the dependency wait on), beyond the rows their registers hold, so
 * that far more of the weight stream is in flight than registers allow.
 * 0 disables it; bytes in [0, 16 MiB]; default 49152 (measured on GB300:
 * 32-64 KB per CTA take the batch-1 layer step from 193 to 172 us; above
 * 128 KB the requested lines start to crowd L2). No counterpart on the pages:
 * a GB300 tuning of the small-matrix kernels [K3 P1§1]. */
dec_status dec_set_l2_ahead(dec_handle* h, int bytes);

/* Force a projection kernel family (DEC_VARIANT_AUTO restores the choice by
 * batch) so that tests can run both families at the same batch. It holds for
 * dec_linear, dec_linear_residual and dec_linear_fp8. */
dec_status dec_set_force_variant(dec_handle* h, int variant);

/* Variant used by the most recent dec_linear / dec_linear_residual /
 * dec_linear_fp8 call on this handle (a dec_variant value; 0 before any call). */
int dec_last_variant(const dec_handle* h);

/* Kernel family of the most recent expert launches (moe_experts,
 * decode_layer): DEC_VARIANT_SMALL_M (batch 1: one token per expert) or
 * DEC_VARIANT_SPLIT_K; 0 before any call. dec_set_force_variant(SPLIT_K)
 * also forces the split-K family for the experts. */
int dec_last_expert_variant(const dec_handle* h);

/* Synchronise the device and read the device error word: DEC_OK if clear,
 * DEC_ERR_TIMEOUT if a kernel gave up a wait since the last check (the word
 * is cleared), DEC_ERR_CUDA if the device reports an error. */
dec_status dec_check_device_error(dec_handle* h);

/* ------------------------------------------------------------------ projections */

/* Workspace bytes that dec_linear / dec_linear_residual need for (M, N, K). */
dec_status dec_linear_workspace_size(const dec_handle* h, int M, int N, int K, size_t* bytes);

/* y[M][N] = x[M][K] W[N][K]^T  (bf16 in, fp32 accumulate, bf16 out).
 * [K3 P1§1], [hu-sum]: the small-matrix kernel at M <= 2 (and up to M = 4
 * for matrices of at most 48 MB, where the split-K kernel's fixed cost per
 * launch dominates), the split-K tcgen05 kernel above (or as forced with
 * dec_set_force_variant). x has row stride ldx >= K elements (ldx = K
 * for a dense matrix; a larger stride reads the leading K columns of a wider
 * activation). 1 <= M <= 64, N >= 1, 8 <= K, K % 8 == 0, ldx % 8 == 0.
 * y must not overlap x or W. */
dec_status dec_linear(dec_handle* h, const dec_bf16* x, int ldx, const dec_bf16* W, dec_bf16* y, int M, int N,
                      int K, void* ws, size_t ws_bytes, cudaStream_t stream);

/* out[M][N] = r[M][N] + x[M][K] W[N][K]^T, the out-projection fused with the
 * residual add [K3 P1§2] (the all-reduce between them has no counterpart on
 * one GPU). fp32 sum, one bf16 rounding. out may alias r exactly. Same shape
 * rules as dec_linear. */
dec_status dec_linear_residual(dec_handle* h, const dec_bf16* x, int ldx, const dec_bf16* W, const dec_bf16* r,
                               dec_bf16* out, int M, int N, int K, void* ws, size_t ws_bytes,
                               cudaStream_t stream);

/* out[M][N] = [r[M][N] +] x[M][K] W[N][K]^T with no workspace argument and
 * no device allocation, for callers that cannot provide scratch memory: for
 * example a plugin running inside a serving runtime whose memory pool owns
 * all device memory and gives plugins no allocator, or a latency-critical
 * caller that must not call cudaMalloc (which can block and synchronise the
 * device). The paper has no counterpart; this is an interface convenience.
 * It runs the split-K tcgen05 kernel of dec_linear with its scratch (10 MiB
 * of split-K partial sums and 4 KiB of tile counters) in one static device
 * array that every GPU loading the library holds until the process exits.
 * - The first call on a device looks up that array's address
 *   (cudaGetSymbolAddress, with the handle's device made current, then the
 *   caller's device restored) and keeps it for the process; make that first
 *   call before any stream capture. A device reset (cudaDeviceReset) after
 *   that first call is not supported: the kept address may no longer be the
 *   array's. A call that fails with DEC_ERR_CUDA drops the kept address, so
 *   the next call looks it up again.
 * - Every call shares the array and it keeps the last call's contents: each
 *   call clears the counters it uses, and calls that overlap on the GPU (for
 *   instance on two streams at once) race on it.
 * - Sizes: the shape rules of dec_linear apply (M outside 1..64, K or ldx
 *   not a multiple of 8 and the like return DEC_ERR_INVALID_ARG); N above
 *   131072, the array's limit, returns DEC_ERR_UNSUPPORTED. r may be NULL;
 *   out may alias r exactly.
 * - Calls no cudaMalloc, cudaFree or other allocating routine. */
dec_status dec_linear_noalloc(dec_handle* h, const dec_bf16* x, int ldx, const dec_bf16* W, const dec_bf16* r,
                              dec_bf16* out, int M, int N, int K, cudaStream_t stream);

/* y[M][H] = x / sqrt(mean(x^2) + eps) * gamma per row (fp32 math, bf16 out).
 * The RMSNorm of the pre-norm decode layer; not named on the pages. y may
 * alias x. 1 <= M <= 64, 8 <= H <= 65536, H % 8 == 0. */
dec_status dec_rmsnorm(dec_handle* h, const dec_bf16* x, const dec_bf16* gamma, dec_bf16* y, int M, int H,
                       float eps, cudaStream_t stream);

/* ------------------------------------------------------------------ router */

dec_status moe_route_topk_workspace_size(const dec_handle* h, int M, int H, int E, size_t* bytes);

/* Router scoring and top-k [K3 P1§3]: logits = x W_r^T (x bf16 [M][H], W_r
 * fp32 [E][H], fp32 math), scores s = sigmoid(logits); per token the k
 * largest scores in descending order, ties to the lower expert id, and
 * weights w_j = s_j / sum of the k selected scores.
 * Outputs: idx int32 [M][k], w fp32 [M][k], scores fp32 [M][E] (scores may be
 * NULL). 1 <= M <= 64, 1 <= k <= 16, k <= E <= 1024, H % 8 == 0. */
dec_status moe_route_topk(dec_handle* h, const dec_bf16* x, const float* Wr, int M, int H, int E, int k,
                          int32_t* idx, float* w, float* scores, void* ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------ experts */

dec_status moe_experts_workspace_size(const dec_handle* h, int M, int k, int E, int H, int I, size_t* bytes);

/* MoE layer body [K3 P1§3]:
 *   out_t = [residual_t +] sum_j w_tj E_{idx_tj}(x_t) [+ S(x_t)]
 * with SwiGLU experts E_e(x) = Wd_e (silu(Wg_e x) * (Wu_e x)).
 * x bf16 [M][H] (the normed hidden state); idx int32 [M][k] in [0, E);
 * w fp32 [M][k]; expert banks Wg, Wu bf16 [E][I][H] and Wd bf16 [E][H][I];
 * shared expert Wg_s, Wu_s bf16 [I][H], Wd_s bf16 [H][I] (all three NULL for
 * none); residual bf16 [M][H] or NULL; out bf16 [M][H] (may alias residual,
 * not x). Each selected expert's weights are read once for all its tokens
 * (at M = 1 each entry is its own problem, so an expert listed twice is read
 * twice). For M >= 2 the shared expert runs on the handle's side stream,
 * overlapped with the routing table and the routed experts, and joins
 * `stream` before return; at M = 1 it is one more problem of the routed
 * launches.
 * The SwiGLU output h is rounded to bf16; everything else stays fp32 until
 * the single bf16 rounding of out.
 * 1 <= M <= 64, 1 <= k <= 16, H and I multiples of 128. */
dec_status moe_experts(dec_handle* h, const dec_bf16* x, const int32_t* idx, const float* w, int M, int k,
                       const dec_bf16* Wg, const dec_bf16* Wu, const dec_bf16* Wd, int E, int H, int I,
                       const dec_bf16* Wg_s, const dec_bf16* Wu_s, const dec_bf16* Wd_s, const dec_bf16* residual,
                       dec_bf16* out, void* ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------ MoE layer */

/* Weights and shape of one MoE layer. */
typedef struct dec_moe_weights {
  int H;                /* hidden size */
  int E;                /* routed experts */
  int k;                /* experts per token */
  int I;                /* expert intermediate size */
  float eps;            /* RMSNorm epsilon (used with gamma) */
  const dec_bf16* gamma;  /* [H] RMSNorm gains applied to the input first, or NULL for none */
  const float* W_r;     /* [E][H] fp32 router */
  const dec_bf16* Wg;   /* [E][I][H] */
  const dec_bf16* Wu;   /* [E][I][H] */
  const dec_bf16* Wd;   /* [E][H][I] */
  const dec_bf16* Wg_s; /* [I][H] or NULL (no shared expert) */
  const dec_bf16* Wu_s; /* [I][H] */
  const dec_bf16* Wd_s; /* [H][I] */
} dec_moe_weights;

dec_status moe_layer_workspace_size(const dec_handle* h, const dec_moe_weights* Wt, int M, size_t* bytes);

/* The MoE layer of a decode step in one call [K3 P1§3, §4]: routing and the
 * experts with the schedule of decode_layer's MoE block:
 *   b       = gamma ? RMSNorm(x; gamma, eps) : x
 *   idx, w  = top-k(sigmoid(b W_r^T)), renormalised
 *   out     = [residual +] sum_j w_j E_idx_j(b) [+ S(b)]
 * x bf16 [M][H]; residual bf16 [M][H] or NULL; out bf16 [M][H] (may alias
 * residual, not x); idx int32 [M][k], w fp32 [M][k] and scores fp32 [M][E]
 * receive the routing when given (each may be NULL). At one token (and two,
 * with a shared expert) the routing, the shared expert's gate/up and the
 * selected experts' gate/up are one launch whose CTAs wait, with the handle's
 * limit, for the routing that one of them publishes; the down projection
 * follows with the combine and the residual. Above, the split-K family runs
 * the shared expert on the handle's side stream. Same shape rules as
 * moe_experts (1 <= M <= 64, 1 <= k <= 16, k <= E <= 1024, H and I multiples
 * of 128). */
dec_status moe_layer(dec_handle* h, const dec_moe_weights* Wt, const dec_bf16* x, const dec_bf16* residual,
                     dec_bf16* out, int M, int32_t* idx, float* w, float* scores, void* ws, size_t ws_bytes,
                     cudaStream_t stream);

/* ------------------------------------------------------------------ decode layer */

/* Weights and shape of one decode layer. */
typedef struct dec_layer_weights {
  int H;     /* hidden size */
  int N_in;  /* width of the attention input projection */
  int K_out; /* input width of the out-projection, K_out <= N_in */
  int E;     /* routed experts */
  int k;     /* experts per token */
  int I;     /* expert intermediate size */
  float eps; /* RMSNorm epsilon */
  const dec_bf16* gamma1; /* [H] */
  const dec_bf16* W_in;   /* [N_in][H] */
  const dec_bf16* W_o;    /* [H][K_out] */
  const dec_bf16* gamma2; /* [H] */
  const float* W_r;       /* [E][H] fp32 */
  const dec_bf16* Wg;     /* [E][I][H] */
  const dec_bf16* Wu;     /* [E][I][H] */
  const dec_bf16* Wd;     /* [E][H][I] */
  const dec_bf16* Wg_s;   /* [I][H] or NULL (no shared expert) */
  const dec_bf16* Wu_s;   /* [I][H] */
  const dec_bf16* Wd_s;   /* [H][I] */
  const void* prefetch_next;   /* optional: weights of the next operator to warm in L2 */
  size_t prefetch_bytes;       /* (multiple of 16; 0 for none) */
} dec_layer_weights;

/* Optional device buffers that receive intermediates of decode_layer (any
 * member may be NULL): h1 bf16 [M][H], idx int32 [M][k], w fp32 [M][k],
 * scores fp32 [M][E]. */
typedef struct dec_layer_trace {
  dec_bf16* h1;
  int32_t* idx;
  float* w;
  float* scores;
} dec_layer_trace;

dec_status decode_layer_workspace_size(const dec_handle* h, const dec_layer_weights* Wt, int M, size_t* bytes);

/* One decode layer in place on h bf16 [M][H]:
 *   a  = RMSNorm(h; gamma1)
 *   y  = a W_in^T                        (small-matrix / split-K by M) [K3 P1§1]
 *   h1 = h + y[:, :K_out] W_o^T           (out-projection + residual)   [K3 P1§2]
 *   b  = RMSNorm(h1; gamma2)
 *   idx, w = top-k(sigmoid(b W_r^T))                                    [K3 P1§3]
 *   h  = h1 + sum_j w_j E_idx_j(b) + S(b)
 * The attention core, which the pages do not define, is read as the identity
 * on the first K_out columns of y. At M = 1 the layer is four launches on
 * `stream`: in-projection with the first RMSNorm, out-projection with the
 * residual, the MoE front (second RMSNorm, router, top-k, routing table, the
 * shared expert's gate/up streamed meanwhile, then the selected experts'
 * gate/up), and the down projection (selected and shared experts) fused with
 * the combine and the residual; M = 2 is the same with two rows. For M >= 3
 * the split-K family runs the shared expert on the handle's side stream
 * [K3 P1§3]. While the router and top-k run, the `prefetch_next` region (if
 * any) is pulled into L2 [K3 P1§4]: by the MoE front's CTAs while they wait
 * for the routing, else by a kernel on a second side stream. trace may be
 * NULL. */
dec_status decode_layer(dec_handle* h, const dec_layer_weights* Wt, dec_bf16* hidden, int M,
                        const dec_layer_trace* trace, void* ws, size_t ws_bytes, cudaStream_t stream);

/* Pull [ptr, ptr + bytes) into L2 on `stream` with an evict-last policy
 * [K3 P1§4]. ptr and bytes multiples of 16. */
dec_status dec_prefetch_l2(dec_handle* h, const void* ptr, size_t bytes, cudaStream_t stream);

/* ------------------------------------------------------------------ attention
 *
 * What stands between the input projection and the out-projection of a decode
 * layer that serves requests: the positions and cache slots of a step's
 * tokens, rotary positions with the write of k and v into a paged cache, and
 * attention over that cache. The sources leave the attention core open; these
 * are the plain operators of a softmax-attention layer.
 *
 * A batch is a list of requests. Request b has own_len[b] tokens of its own
 * in the cache after this step, the last row_start[b + 1] - row_start[b] of
 * which are this step's rows; before them come prefix_len tokens that all
 * requests of the batch share. A request may have no rows (a finished one),
 * and rows at and behind row_start[requests] belong to none (padding).
 * Lengths, tables and slots are device memory, so a captured graph can be
 * replayed with new ones. int32 arrays need 4-byte alignment only. */

/* The paged key / value cache of one layer. Block i holds
 * [kv_heads][block_size][head_dim] values at k + i * block_stride (and at
 * v + i * block_stride); slot s is token s % block_size of block
 * s / block_size. k and v may interleave in one pool (a larger stride). */
typedef struct dec_kv_cache {
  dec_bf16* k;
  dec_bf16* v;
  int64_t block_stride; /* elements; at least kv_heads * block_size * head_dim, a multiple of 8 */
  int blocks;           /* blocks * block_size < 2^31 */
  int block_size;       /* 16, 32, 64 or 128 */
  int kv_heads;         /* 1..128 */
  int head_dim;         /* 64 or 128 */
} dec_kv_cache;

/* The requests of one step, as attention reads them. */
typedef struct dec_batch {
  int requests;               /* 1..64 */
  int max_new;                /* at least the rows of any one request, 1..64 */
  const int32_t* row_start;   /* [requests + 1] first row of each request, not decreasing */
  const int32_t* own_len;     /* [requests] own tokens in the cache, this step's included */
  const int32_t* block_table; /* [requests][max_blocks] cache blocks of the own tokens, in order */
  int max_blocks;             /* at least 1; max_blocks * block_size <= 2^31 - 256 */
  const int32_t* prefix_table; /* [ceil(prefix_len / block_size)] blocks of the shared prefix; NULL if none */
  int prefix_len;             /* 0: no shared prefix; at most 2^31 - 256 */
} dec_batch;

/* Outputs of dec_batch_tables (device memory). */
typedef struct dec_step_tables {
  int32_t* row_start; /* [requests + 1] */
  int32_t* own_len;   /* [requests]; may be ctx_len itself */
  int32_t* positions; /* [rows] */
  int32_t* slots;     /* [rows] */
  int32_t* left;      /* [2] */
} dec_step_tables;

/* Positions, slots and block-table entries of one step, built on the GPU from
 * the requests' lengths. Request b holds ctx_len[b] own tokens in the cache
 * and gets new_len[b] more (negative values count as 0):
 *   row_start = exclusive running sum of new_len, held at `rows`
 *   own_len   = ctx_len + the request's rows
 *   position of row i of request b = position_offset + ctx_len[b] + i
 * A request whose rows reach past its ceil(ctx_len / block_size) held blocks
 * gets blocks from the free list free_blocks[0 .. *free_count), taken from its
 * end, requests in order, and they are entered in its row of
 * block_table [requests][max_blocks]; the entries it holds stay as they are.
 *   slots[t] = block_table[b][j / block_size] * block_size + j % block_size
 * for row t's own token j, and -1 where it has no block: the free list was
 * used up (such entries become -1), j is past max_blocks blocks, or the held
 * entry is negative. Rows behind the last request get slot -1 and position 0.
 *   left[0] = free blocks that remain (pass it as the next step's free_count,
 *             it may be the same memory), left[1] = rows of requests that got
 *             no slot
 * A request that ends gives its blocks back when the caller puts them behind
 * the remaining ones in free_blocks and raises the count. Rows that new_len
 * gives past `rows` are left out (row_start is held at rows). One launch, no
 * workspace; the results depend on the inputs alone.
 * 1 <= requests <= 1024, 1 <= rows <= 2^20, block_size 16, 32, 64 or 128,
 * 1 <= max_blocks <= 2^24, position_offset >= 0. Apart from the pairs named
 * above, no output may overlap an input. */
dec_status dec_batch_tables(dec_handle* h, const int32_t* ctx_len, const int32_t* new_len, int requests,
                            const int32_t* free_blocks, const int32_t* free_count, int32_t* block_table,
                            int max_blocks, int block_size, int position_offset, int rows,
                            const dec_step_tables* out, cudaStream_t stream);

/* How rotary frequencies are stretched for contexts longer than the original
 * length L, by a factor f >= 1, for pairs i of R = rotary_dim:
 * f_i = base^(-2 i / R) radians a position, and then
 *  NONE:   f_i
 *  LINEAR: f_i / f
 *  NTK:    f_i of base * f^(R / (R - 2))
 *  BANDS:  k f_i + (1 - k) f_i / f, k = clamp((turns_i - low) / (high - low)),
 *          turns_i = L f_i / 2 pi: pairs that turn fast are kept, slow ones
 *          divided, a blend by turns between
 *  YARN:   the same blend as a ramp over the pair's index i, from
 *          floor(c(high)) to ceil(c(low)), c(t) = R ln(L / 2 pi t) / (2 ln base),
 *          held in [0, R - 1] (Peng et al., "YaRN", 2023); its factor on the
 *          logits, 0.1 ln f + 1 on q and k each, is dec_rope's magnitude */
typedef enum dec_rope_scaling {
  DEC_ROPE_NONE = 0,
  DEC_ROPE_LINEAR = 1,
  DEC_ROPE_NTK = 2,
  DEC_ROPE_BANDS = 3,
  DEC_ROPE_YARN = 4
} dec_rope_scaling;

/* Write the rotary_dim / 2 phase steps that dec_rope_append reads: step i is
 * the fraction of a turn that pair i moves per position, f_i / 2 pi, in units
 * of 2^-64 turns (computed in 64-bit floating point). Position times step,
 * modulo 2^64, is then the angle modulo a turn at any int32 position, exact
 * to 2^-53 of the step's own rounding, with no range reduction left.
 * rotary_dim a multiple of 16 in [16, 128], base > 1, factor >= 1;
 * original_len > 0 and 0 < low < high are read by BANDS and YARN only. */
dec_status dec_rope_phases(dec_handle* h, uint64_t* phases, int rotary_dim, double base, int scaling, double factor,
                           double original_len, double low, double high, cudaStream_t stream);

typedef struct dec_rope {
  int rotary_dim;         /* leading elements of each head that turn: a multiple of 16 up to head_dim; 0: none */
  int interleaved;        /* 0: pairs (i, i + rotary_dim / 2); 1: pairs (2 i, 2 i + 1) */
  float magnitude;        /* factor on cos and sin (1 unless the scaling asks for another), finite */
  const uint64_t* phases; /* [rotary_dim / 2] from dec_rope_phases, 16-byte aligned; NULL if rotary_dim is 0 */
} dec_rope;

/* Turn q and k by their rows' positions and write k and v into the cache:
 *   q_out[t] = R(positions[t]) q[t]          (all `rows` rows)
 *   cache.k[slots[t]] = R(positions[t]) k[t], cache.v[slots[t]] = v[t]
 * where R turns each pair (a, b) of the first rotary_dim elements of a head
 * to (a c - b s, b c + a s), c and s being magnitude times cos and sin, and
 * leaves the rest of the head. fp32 math, one bf16 rounding. Rows whose slot
 * is negative or past the cache write no k and v. No two rows may have the
 * same slot. q [rows][q_heads * head_dim] with row stride ldq, and k, v
 * [rows][kv_heads * head_dim] with row strides ldk, ldv, may be columns of
 * one projection's output; q_out (row stride ldqo) may be q itself with the
 * same stride. q and q_out both NULL (q_heads 0): only the cache is written.
 * 1 <= rows <= 2^20, q_heads <= 1024, strides multiples of 8. */
dec_status dec_rope_append(dec_handle* h, const dec_rope* rope, const dec_bf16* q, int64_t ldq, const dec_bf16* k,
                           int64_t ldk, const dec_bf16* v, int64_t ldv, dec_bf16* q_out, int64_t ldqo, int rows,
                           int q_heads, const int32_t* positions, const int32_t* slots, const dec_kv_cache* cache,
                           cudaStream_t stream);

dec_status dec_attention_workspace_size(const dec_handle* h, int M, int q_heads, const dec_kv_cache* cache,
                                        const dec_batch* batch, size_t* bytes);

/* Attention of a step's rows over the cache: for row i of the n of request b
 * and query head g (key / value head g / (q_heads / kv_heads)),
 *   out = sum_j p_j v_j, p = softmax_j(scale q . k_j)
 * over the prefix_len shared tokens and the own tokens
 * j < own_len[b] - n + i + 1: each row sees the rows before it. The shared
 * prefix is read once for all rows, not once a request. Tokens in a block
 * whose table entry is outside [0, blocks), or past max_blocks blocks, are
 * not there. A row that sees no token gets zeros; rows of no request are left
 * as they were. A row follows from the tokens that it sees alone: the rows
 * behind it and places of the cache that hold none of these tokens may hold
 * infinities and NaN.
 * q [M][q_heads * head_dim] with row stride ldq, out the same with ldo; out
 * must not overlap q. 1 <= M <= 64, q_heads a multiple of kv_heads, at most
 * 1024 in all and 128 to a key head, scale in [1e-30, 1e30]. Scores, softmax
 * statistics and sums are fp32; the weights p, up to a factor that a row's
 * keys share, are rounded to bf16 for the product with v. */
dec_status dec_attention(dec_handle* h, const dec_bf16* q, int64_t ldq, const dec_kv_cache* cache,
                         const dec_batch* batch, float scale, dec_bf16* out, int64_t ldo, int M, int q_heads,
                         void* ws, size_t ws_bytes, cudaStream_t stream);

/* The attention core of one decode layer. */
typedef struct dec_layer_attention {
  int q_heads;               /* q_heads * head_dim = K_out */
  float scale;               /* factor on the scores, in [1e-30, 1e30] */
  const dec_rope* rope;      /* rotary positions, or NULL for none */
  const dec_kv_cache* cache; /* the layer's cache */
  const dec_batch* batch;
  const int32_t* positions;  /* [M], from dec_batch_tables */
  const int32_t* slots;      /* [M] */
} dec_layer_attention;

dec_status decode_layer_attention_workspace_size(const dec_handle* h, const dec_layer_weights* Wt,
                                                 const dec_layer_attention* A, int M, size_t* bytes);

/* decode_layer with attention in place of the identity:
 *   y = RMSNorm(h; gamma1) W_in^T = [q | k | v | rest],
 *       q_heads, kv_heads and kv_heads heads of head_dim columns
 *   q, k turned by their positions, k and v written to the cache
 *   h1 = h + attention(q) W_o^T, and the rest of the layer as it is there.
 * Wt->K_out = q_heads * head_dim, Wt->N_in >= (q_heads + 2 kv_heads) *
 * head_dim. The rows' own tokens must be counted in batch->own_len already (as
 * dec_batch_tables does). Rows of no request pass with an attention output of
 * zero. Everything else (workspace, trace, prefetch) as in decode_layer; the
 * shape that a workspace is zeroed for includes q_heads, kv_heads, head_dim
 * and whether there is a prefix. */
dec_status decode_layer_attention(dec_handle* h, const dec_layer_weights* Wt, const dec_layer_attention* A,
                                  dec_bf16* hidden, int M, const dec_layer_trace* trace, void* ws, size_t ws_bytes,
                                  cudaStream_t stream);

/* ------------------------------------------------------------------ 8-bit weights and rows
 *
 * The layer's products with half the weight bytes. An e4m3 number (1 sign, 4
 * exponent, 3 mantissa bits, largest value 448, no infinities) stands for
 * itself times a 32-bit scale:
 *   weights W[N][K]:  one scale for each block of 128 x 128,
 *                     scales[ceil(N / 128)][ceil(K / 128)]
 *   rows x[M][K]:     one for each 128 values of a row, from its start
 * the last blocks of a row or matrix being what is left. A group is quantised
 * by its largest absolute value m: scale = m / 448, q = e4m3(value * (448 / m)),
 * nearest-even; a group with m < 2^-116 is zeros with scale 0. A group that
 * holds a NaN or an infinity has it as its scale, so what reads it becomes NaN.
 * Rows and reduction lengths K are multiples of 16 here. */

typedef uint8_t dec_e4m3; /* bit pattern of an e4m3 value */

/* Rows of 8-bit values: row t at q + t * ldq, its scales at scales + t * lds. */
typedef struct dec_fp8_rows {
  dec_e4m3* q;   /* 16-byte aligned */
  int64_t ldq;   /* elements, a multiple of 16, at least the width */
  float* scales; /* 4-byte aligned */
  int64_t lds;   /* at least ceil(width / 128) */
} dec_fp8_rows;

/* An 8-bit weight matrix [N][K] and its block scales, both without gaps. */
typedef struct dec_fp8_weight {
  const dec_e4m3* q;   /* 16-byte aligned */
  const float* scales; /* 4-byte aligned */
} dec_fp8_weight;

/* A bf16 weight matrix [N][K] to 8 bits with block scales, for load time. A
 * bank of E experts of I rows is one matrix of E I rows if I is a multiple of
 * 128. 1 <= N <= 2^32, K a multiple of 16 in [16, 65536]. */
dec_status dec_quant_weight(dec_handle* h, const dec_bf16* W, int64_t N, int K, dec_e4m3* q, float* scales,
                            cudaStream_t stream);

/* The residual's addition, the RMSNorm and its rows in 8 bits, in one pass:
 *   a = residual ? bf16(x + residual) : x       -> sum, if given
 *   b = gamma ? a / sqrt(mean(a^2) + eps) * gamma : a   (fp32) -> y in bf16, if given
 *   out = b in 8 bits, quantised from fp32
 * All bf16 rows have H contiguous values and a row stride in elements, a
 * multiple of 8. sum (only with a residual) may be x or residual itself, y too,
 * with the same stride; apart from that no output overlaps an input or another
 * output. y has the bits that dec_rmsnorm gives for a. gamma NULL quantises
 * rows that need no norm, such as the attention's output.
 * 1 <= M <= 2^20, H a multiple of 16 in [16, 65536]. */
dec_status dec_rmsnorm_quant(dec_handle* h, const dec_bf16* x, int64_t ldx, const dec_bf16* residual, int64_t ldr,
                             const dec_bf16* gamma, float eps, dec_bf16* sum, int64_t lds, dec_bf16* y, int64_t ldy,
                             const dec_fp8_rows* out, int M, int H, cudaStream_t stream);

dec_status dec_linear_fp8_workspace_size(const dec_handle* h, int M, int N, int K, size_t* bytes);

/* y[M][N] = [residual[M][N] +] x[M][K] W[N][K]^T on 8-bit rows and weights.
 * Within a block of 128 the products and their sum are fp32; the block's sum is
 * scaled and added to the total in fp32, and y is rounded once. y and residual
 * have row strides ldy, ldr >= N in elements (any, 2-byte aligned); y may be
 * residual itself with the same stride and overlaps nothing else.
 * Kernel families as for dec_linear: SMALL_M streams the weights past the rows
 * (M <= 16), SPLIT_K is the tcgen05 kernel; AUTO takes the first up to M = 8, and
 * up to 16 for weights of at most 64 MB. Rows that the first's shared memory does
 * not hold (16 of 8192 values fit, 8 of 16384, 2 of 65536) take the second, forced
 * or not. Weights may be read before the launch's
 * dependency wait, as static data; dec_quant_weight just before is safe.
 * The workspace (none for SMALL_M) is zeroed before its first use and then serves
 * calls of any shape, one at a time, also after DEC_ERR_TIMEOUT; its size depends
 * on the forced family.
 * 1 <= M <= 2^20 (prompts too), 1 <= N <= 2^20, K a multiple of 16 in
 * [16, 65536]. */
dec_status dec_linear_fp8(dec_handle* h, const dec_fp8_rows* x, const dec_fp8_weight* W, const dec_bf16* residual,
                          int64_t ldr, dec_bf16* y, int64_t ldy, int M, int N, int K, void* ws, size_t ws_bytes,
                          cudaStream_t stream);

/* Weights of an MoE layer's experts in 8 bits: gate, up [E][I][H] and down
 * [E][H][I] with scales [E][I / 128][H / 128] and [E][H / 128][I / 128]; the
 * shared expert's are one expert's, or all NULL. */
typedef struct dec_moe_fp8_weights {
  int H; /* hidden size, a multiple of 128 */
  int E; /* routed experts, at most 1024 */
  int I; /* expert intermediate size, a multiple of 128 */
  dec_fp8_weight gate, up, down;
  dec_fp8_weight gate_s, up_s, down_s;
} dec_moe_fp8_weights;

dec_status moe_experts_fp8_workspace_size(const dec_handle* h, const dec_moe_fp8_weights* Wt, int M, int k,
                                          size_t* bytes);

/* moe_experts on 8-bit rows and weights:
 *   out_t = [residual_t +] sum_j w_tj E_{idx_tj}(x_t) [+ S(x_t)],
 *   E(x) = Wd q(silu(Wg x) * (Wu x))
 * where q quantises the inner row from fp32 by groups of 128, as
 * dec_rmsnorm_quant does. Everything else is fp32 until out is rounded to bf16.
 * x [M][H]; idx int32 [M][k] and w fp32 [M][k] as from moe_route_topk; an entry
 * whose id is outside [0, E) is left out. residual bf16 [M][H] or NULL; out bf16
 * [M][H], which may be residual itself and overlaps nothing else. Each problem
 * (an expert with up to 8 or 16 of its tokens) streams the expert's weights once.
 * The workspace needs no particular contents. 1 <= M <= 64, 1 <= k <= 16, H and I up to 16384
 * (else DEC_ERR_UNSUPPORTED). */
dec_status moe_experts_fp8(dec_handle* h, const dec_fp8_rows* x, const int32_t* idx, const float* w, int M, int k,
                           const dec_moe_fp8_weights* Wt, const dec_bf16* residual, dec_bf16* out, void* ws,
                           size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------ measurement */

/* Per-kernel timing record returned by dec_profile_read. */
typedef struct dec_kernel_time {
  char name[32];   /* kernel tag, e.g. "in_proj", "gate_up", "shared_down" */
  int launches;    /* launches since the last read */
  double total_ms; /* summed device time of those launches */
} dec_kernel_time;

/* Enable (1) or disable (0) per-kernel timing: every kernel launch is then
 * bracketed by CUDA events on the stream it is launched on. The events
 * separate kernels, so programmatic dependent launch overlap is lost while
 * profiling is on; use it for per-kernel durations, not for step times. */
dec_status dec_set_profiling(dec_handle* h, int enable);

/* Synchronise, then aggregate the timing records by kernel tag into
 * out[0 .. capacity) (*count receives the number of tags) and clear them. */
dec_status dec_profile_read(dec_handle* h, dec_kernel_time* out, int capacity, int* count);

/* Number of kernels this handle has launched since it was created. */
uint64_t dec_launch_count(const dec_handle* h);

/* ------------------------------------------------------------------ test hooks */

/* Launch a kernel whose mbarrier wait can never complete; it must give up
 * after the handle's wait limit and set the device error word. Used to test
 * that timeouts surface as DEC_ERR_TIMEOUT with the context still usable. */
dec_status dec_test_wait_timeout(dec_handle* h, cudaStream_t stream);

/* Run the MoE front launch (tokens: 1, or 2 for the few-token kernel) on a
 * small zeroed problem whose routing hand-off can never complete (its arrival
 * counter starts past the grid size), so the routing flag is never set: every
 * CTA's wait for it must give up after the handle's wait limit and set the
 * device error word. Allocates and frees its own buffers and synchronises
 * `stream`. Used to test that the routing wait surfaces as DEC_ERR_TIMEOUT
 * with the context still usable. tokens outside {1, 2}: DEC_ERR_INVALID_ARG. */
dec_status dec_test_routing_wait_timeout(dec_handle* h, int tokens, cudaStream_t stream);

/* 1 (default): decode_layer and moe_layer use the MoE front launches at one
 * and two tokens when there is a shared expert (routing, the shared expert's
 * gate/up and the selected experts' gate/up in one launch). 0: they use the
 * launches taken where a front does not apply (no shared expert, or shapes
 * outside its limits): the routing launch, then the grouped gate/up with the
 * shared expert as one more problem, then the down projection. Both compute
 * the same layer; the hook lets tests run the second path with a shared
 * expert. */
dec_status dec_test_set_moe_front(dec_handle* h, int enable);

/* How the split-K kernel finishes a tile split between CTAs (a tile's partial
 * sums from several CTAs' ranges of k). 0 (default): the CTA holding the
 * first piece waits a bounded time for the others, then adds all pieces in k
 * order from shared memory; past the bound it publishes its piece, and the
 * CTA that completes the count finishes the tile. 1: every CTA publishes its
 * piece at once, so the tile is always finished by the CTA that completes the
 * count (from shared memory when that CTA is at the end of its range). 2: as
 * 1, and the finishing CTA always reads the pieces with batched loads from
 * L2. All three add the same fp32 partials in the same k order, so they give
 * the same bits; the hook lets tests check that. Other values:
 * DEC_ERR_INVALID_ARG. */
dec_status dec_test_set_engine_finish(dec_handle* h, int mode);

/* every > 0: in the tcgen05 kernel of dec_linear_fp8 the CTAs whose index is a
 * multiple of `every` act as if their first wait had run past the limit: they
 * set the device error word, drain what they have in flight and leave. 0
 * (default): none. Used to test that a call whose waits ran out in part of its
 * CTAs leaves its workspace ready. */
dec_status dec_test_set_linear_fp8_give_up(dec_handle* h, int every);

/* Hold `ctas` SMs (1 <= ctas <= the device's SM count) for hold_ns
 * nanoseconds (at most 2 s) with a kernel on `stream`: one CTA per SM that
 * takes the whole per-block shared memory, so nothing else fits beside it,
 * and sleeps on the global timer. It writes nothing. Used to test that the
 * MoE fronts complete when another stream's kernel holds part of the SMs, so
 * that not all of their CTAs can be resident at once. */
dec_status dec_test_occupy_sms(dec_handle* h, int ctas, uint64_t hold_ns, cudaStream_t stream);

/* Copy `bytes` from src to dst on `stream` after spinning for delay_ns
 * (bounded by the clock): a slow producer for ordering tests of the
 * programmatic-dependent-launch path. */
dec_status dec_test_delayed_copy(dec_handle* h, void* dst, const void* src, size_t bytes, uint64_t delay_ns,
                                 cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DECODE_H */
