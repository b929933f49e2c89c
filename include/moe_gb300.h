/*
 * moe_gb300.h — C ABI of the routed fused-MoE expert GEMM for GB300 (sm_103a).
 *
 * Token rows arrive grouped by expert and padded to 128-row blocks, described
 * by four int32 dispatch tables.  For every valid row p of expert e
 *
 *     up_logits[p, :] = fp16( silu(x[p]·gate_w[e]ᵀ) ⊙ (x[p]·up_w[e]ᵀ) )
 *     out[p, :]       = fp16( (up_logits[p]·down_w[e]ᵀ) · routed_expert_weights[c] )
 *
 * with fp32 accumulation, c = group_offsets[e] + (p - group_padded_offsets[e])
 * the row's compact index, and padding rows neither computed nor written.
 * Source: "Fused MoE GEMM 提交说明", §算子来源 (the expert MLP), §实现要点
 * (padded vs compact indexing, padding rows untouched), §完整算子代码 (the
 * run_kernel argument list, block_token = 128, fp16 data with fp32
 * accumulation, up_logits as an fp16 workspace); "moe_dispatch_contract.py"
 * (TileLang tutorial, ch. 18) for the four tables; "MetaX-TileLang工具链"
 * §1.9 for the two launches and their arguments.
 *
 * Conventions for every entry point:
 *   - All array arguments are DEVICE pointers owned by the caller.  The library
 *     never allocates, frees or keeps a pointer after the call returns.
 *   - fp16 data is passed as `uint16_t` bit patterns (IEEE binary16).
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every
 *     call is asynchronous: it validates its arguments on the host, enqueues
 *     kernels and returns without synchronising.
 *   - A negative return value (MOE_ERR_*) means nothing was enqueued.
 *   - `status_dev` (nullable) is a device int32 into which kernels OR
 *     MOE_DEV_* bits when they meet inconsistent data (an expert id or table
 *     entry out of range, a bounded wait that ran out).  Offending work items
 *     are skipped; kernels never trap.  The caller zeroes it and reads it back.
 *   - Shapes are limited to hidden % 128 == 0, intermediate % 128 == 0,
 *     block_token == 128, 1 <= n_experts <= MOE_MAX_EXPERTS,
 *     num_blocks_m <= MOE_MAX_BLOCKS, unless a call says otherwise.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t moe_status_t;

#define MOE_OK            0
#define MOE_ERR_NULL     -1  /* a required pointer is NULL                          */
#define MOE_ERR_SHAPE    -2  /* a size is negative, inconsistent or not the multiple asked for */
#define MOE_ERR_ALIGN    -3  /* a pointer is not 16-byte aligned (TMA needs it)      */
#define MOE_ERR_BLOCK    -4  /* block_token != 128                                   */
#define MOE_ERR_DEVICE   -5  /* no usable sm_103 device / driver entry point         */
#define MOE_ERR_LAUNCH   -6  /* a kernel launch failed (cudaGetLastError)            */
#define MOE_ERR_LIMIT    -7  /* n_experts or num_blocks_m above the library limits   */
#define MOE_ERR_WORKSPACE -8 /* workspace missing or smaller than required           */
#define MOE_ERR_STATIC_WORKSPACE -9 /* problem larger than the library's fixed workspace */

/* Bits OR-ed into *status_dev by kernels. */
#define MOE_DEV_BAD_EXPERT_ID 0x1  /* a topk id outside [0, n_experts)                 */
#define MOE_DEV_BAD_TABLE     0x2  /* a table entry points outside its array           */
#define MOE_DEV_TIMEOUT       0x4  /* a bounded pipeline wait ran out; tiles skipped    */
#define MOE_DEV_DEBUG_CHECK   0x8  /* MOE_DEBUG builds only: a kernel's own check of an
                                      index, coordinate or shared-memory canary failed */

#define MOE_BLOCK_TOKEN  128
#define MOE_MAX_EXPERTS  1024
#define MOE_MAX_BLOCKS   16384

/* Version of this ABI (bumped on any incompatible change). */
int32_t moe_abi_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char* moe_status_string(moe_status_t status);

/* Number of 128-row blocks of the padded layout:
 *     ceil(pairs / block_token) + n_experts
 * ("moe_dispatch_contract.py", build_contract step 4; "MetaX-TileLang工具链"
 * §1.9: M = ceil(group_sum / block_token) + group_count).  Every expert owns at
 * least one block because of the "+1" padding rule, so this bounds the padded
 * row count.  Returns -1 for negative arguments or block_token <= 0. */
int64_t moe_num_blocks(int64_t pairs, int32_t n_experts, int32_t block_token);

/* Build the four dispatch tables on the GPU from routing choices
 * ("moe_dispatch_contract.py", docstring and build_contract).
 *   topk_ids              [n_tokens, top_k] int32, row-major; the flat pair
 *                         index is t*top_k + j.  Ids must lie in [0, n_experts).
 *   group_sizes           [n_experts]   out: pairs routed to each expert
 *   group_offsets         [n_experts+1] out: exclusive prefix sum of the sizes
 *                         (compact rows); entry n_experts = total pairs
 *   group_padded_offsets  [n_experts+1] out: exclusive prefix sum of
 *                         ceil((size+1)/block_token)*block_token (padded rows);
 *                         entry n_experts = total padded rows
 *   group_idx_for_bx      [num_blocks_m] out: for block bx, the last expert e
 *                         with group_padded_offsets[e] <= bx*block_token
 *   num_blocks_m          must equal moe_num_blocks(n_tokens*top_k, n_experts, block_token)
 * Out-of-range ids are not counted and set MOE_DEV_BAD_EXPERT_ID.  One kernel
 * launch; no workspace. */
moe_status_t moe_build_dispatch(const int32_t* topk_ids, int64_t n_tokens, int32_t top_k,
                                int32_t n_experts, int32_t block_token,
                                int32_t* group_sizes, int32_t* group_offsets,
                                int32_t* group_padded_offsets, int32_t* group_idx_for_bx,
                                int64_t num_blocks_m, int32_t* status_dev, void* stream);

/* The fused forward: phase 1 (grouped gate+up GEMM, SiLU·up epilogue into the
 * fp16 up_logits workspace) then phase 2 (grouped down GEMM, routed weight
 * applied to the fp32 accumulator, fp16 store) — "Fused MoE GEMM 提交说明",
 * §完整算子代码, the page's run_kernel contract plus the explicit up_logits
 * argument of "MetaX-TileLang工具链" §1.9.
 *   stacked_expert_tokens [total_padded_tokens, hidden] fp16, padded rows
 *   gate_w, up_w          [n_experts, intermediate, hidden] fp16
 *   down_w                [n_experts, hidden, intermediate] fp16
 *   routed_expert_weights [total_valid_tokens] fp32, compact (expert-sorted) order
 *                         (may be NULL when total_valid_tokens == 0)
 *   group_*               the four tables above (only entries [0, n_experts) of
 *                         group_offsets / group_padded_offsets are read)
 *   up_logits             [total_padded_tokens, intermediate] fp16 workspace
 *   out                   [total_padded_tokens, hidden] fp16
 * Requirements: total_padded_tokens >= num_blocks_m*128; hidden and
 * intermediate multiples of 128; every pointer 16-byte aligned.  Rows that are
 * not valid rows of some block are never written, in up_logits or out.
 * Two kernel launches on `stream` (the second with programmatic dependent
 * launch); no workspace beyond up_logits. */
moe_status_t moe_fused_forward(const uint16_t* stacked_expert_tokens, int64_t total_padded_tokens,
                               int32_t hidden,
                               const uint16_t* gate_w, const uint16_t* up_w, const uint16_t* down_w,
                               int32_t n_experts, int32_t intermediate,
                               const float* routed_expert_weights, int64_t total_valid_tokens,
                               const int32_t* group_sizes, const int32_t* group_offsets,
                               const int32_t* group_padded_offsets,
                               const int32_t* group_idx_for_bx, int64_t num_blocks_m,
                               uint16_t* up_logits, uint16_t* out,
                               int32_t* status_dev, void* stream);

/* Workspace bytes moe_pack_routed needs for `pairs` (token, expert) pairs
 * (per-chunk expert histograms and every pair's rank inside its chunk).
 * Returns -1 for invalid arguments. */
int64_t moe_pack_workspace_bytes(int64_t pairs, int32_t n_experts);

/* Pack: place every (token, expert) pair in the grouped, padded layout that
 * moe_fused_forward reads.  Pairs are stably sorted by expert
 * ("moe_dispatch_contract.py", build_contract), so the pair of rank r inside
 * expert e (counting pairs in flat order t*top_k + j) goes to padded row
 * group_padded_offsets[e] + r and compact index group_offsets[e] + r
 * ("Fused MoE GEMM 提交说明", §实现要点).
 *   topk_ids, topk_weights  [n_tokens, top_k] int32 / fp32 (weights may be NULL
 *                           when routed_expert_weights is NULL)
 *   x_tokens                [n_tokens, hidden] fp16 (may be NULL when
 *                           stacked_expert_tokens is NULL)
 *   group_offsets, group_padded_offsets  the tables of moe_build_dispatch
 *   stacked_expert_tokens   out, nullable: [total_padded_tokens, hidden]; row
 *                           pair_padded_rows[f] receives x_tokens[f / top_k];
 *                           padding rows are not written
 *   routed_expert_weights   out, nullable: [n_tokens*top_k] fp32, compact order
 *   pair_padded_rows        out: [n_tokens, top_k] int32 padded row of every
 *                           pair (-1 for an id outside [0, n_experts))
 *   workspace               device scratch of moe_pack_workspace_bytes() bytes
 * Three kernel launches; an out-of-range id sets MOE_DEV_BAD_EXPERT_ID. */
moe_status_t moe_pack_routed(const int32_t* topk_ids, const float* topk_weights, int64_t n_tokens,
                             int32_t top_k, int32_t n_experts, const uint16_t* x_tokens, int32_t hidden,
                             const int32_t* group_offsets, const int32_t* group_padded_offsets,
                             int64_t total_padded_tokens, uint16_t* stacked_expert_tokens,
                             float* routed_expert_weights, int32_t* pair_padded_rows,
                             void* workspace, size_t workspace_bytes, int32_t* status_dev, void* stream);

/* Combine: y[t, :] = fp16( sum over j = 0..top_k-1, in that order, of
 * out[pair_padded_rows[t*top_k + j], :] ) with the sum in fp32 and one
 * round-to-nearest-even.  The pages combine with a PyTorch scatter_reduce
 * ("MetaX-TileLang工具链", §2.7); the routed weight is already inside `out`.
 *   out               [total_padded_tokens, hidden] fp16 (moe_fused_forward's)
 *   pair_padded_rows  [n_tokens, top_k] int32 (moe_pack_routed's); negative
 *                     entries are skipped
 *   y                 out: [n_tokens, hidden] fp16
 * One kernel launch. */
moe_status_t moe_combine_routed(const uint16_t* out, int64_t total_padded_tokens, int32_t hidden,
                                const int32_t* pair_padded_rows, int64_t n_tokens, int32_t top_k,
                                uint16_t* y, void* stream);

#define MOE_ROUTER_MAX_EXPERTS 256
#define MOE_ROUTER_MAX_TOPK    16

/* Router ("MetaX-TileLang工具链", §2.4: logits = W_g(x), scores =
 * softmax(logits), topk_scores, topk_indices = topk(scores)).
 *   x_tokens      [n_tokens, hidden] fp16
 *   router_w      [n_experts, hidden] fp16 (W_g; a logit is a row of W_g
 *                 dotted with the token, accumulated in fp32)
 *   topk_ids      out: [n_tokens, top_k] int32, the top_k experts by logit in
 *                 descending order; equal logits: the lower expert index first
 *   topk_weights  out: [n_tokens, top_k] fp32, their softmax probabilities over
 *                 all n_experts (not renormalised over the k)
 * Limits: hidden % 128 == 0, n_experts <= MOE_ROUTER_MAX_EXPERTS, top_k <=
 * min(n_experts, MOE_ROUTER_MAX_TOPK).  One kernel launch: a tcgen05 MMA tile
 * of 128 tokens x all experts per cluster of 1-8 CTAs (hidden split over the
 * cluster when there are fewer tiles than SMs), softmax and top-k in its
 * epilogue.  Every wait inside it is bounded (2 s); one that runs out sets
 * MOE_DEV_TIMEOUT in status_dev (nullable) and leaves the outputs invalid. */
moe_status_t moe_router_topk(const uint16_t* x_tokens, int64_t n_tokens, int32_t hidden,
                             const uint16_t* router_w, int32_t n_experts, int32_t top_k,
                             int32_t* topk_ids, float* topk_weights, int32_t* status_dev, void* stream);

/* moe_router_topk that also keeps the logits, for the losses and gradients below:
 *   logits        out, nullable: [n_tokens, n_experts] fp32, 16-byte aligned */
moe_status_t moe_router_topk_logits(const uint16_t* x_tokens, int64_t n_tokens, int32_t hidden,
                                    const uint16_t* router_w, int32_t n_experts, int32_t top_k, int32_t* topk_ids,
                                    float* topk_weights, float* logits, int32_t* status_dev, void* stream);

/* Flags of moe_fused_forward_ex. */
#define MOE_RUN_PHASE1   0x1u  /* gate+up GEMM and SiLU·up epilogue into up_logits   */
#define MOE_RUN_PHASE2   0x2u  /* down GEMM and routed-weight epilogue into out       */
#define MOE_NO_PDL       0x4u  /* launch phase 2 without programmatic dependent launch */
/* Test of the failure path: phase 1's MMA issuer skips its first "accumulator
 * ready" signal, so an epilogue wait runs out after its bound (2 s); the
 * kernel then stops, frees its resources and reports MOE_DEV_TIMEOUT in
 * status_dev.  The outputs of such a call are not valid. */
#define MOE_TEST_DROP_SIGNAL 0x100u

/* moe_fused_forward with a choice of phases: `flags` is a combination of
 * MOE_RUN_PHASE1 / MOE_RUN_PHASE2 (at least one) and optionally MOE_NO_PDL.
 * Running phase 2 alone reads up_logits as left by an earlier phase 1 on the
 * same tables (for example to time each phase by itself).  Same arguments,
 * requirements and errors as moe_fused_forward, which is this call with
 * flags = MOE_RUN_PHASE1 | MOE_RUN_PHASE2. */
moe_status_t moe_fused_forward_ex(const uint16_t* stacked_expert_tokens, int64_t total_padded_tokens,
                                  int32_t hidden,
                                  const uint16_t* gate_w, const uint16_t* up_w, const uint16_t* down_w,
                                  int32_t n_experts, int32_t intermediate,
                                  const float* routed_expert_weights, int64_t total_valid_tokens,
                                  const int32_t* group_sizes, const int32_t* group_offsets,
                                  const int32_t* group_padded_offsets,
                                  const int32_t* group_idx_for_bx, int64_t num_blocks_m,
                                  uint16_t* up_logits, uint16_t* out,
                                  int32_t* status_dev, void* stream, uint32_t flags);

/* Workspace bytes of moe_fused_forward_single_launch (one int32 counter per
 * 128-row block, rounded up).  Returns -1 for a negative argument. */
int64_t moe_single_launch_workspace_bytes(int64_t num_blocks_m);

/* moe_fused_forward with both phases in ONE persistent launch (same
 * arguments, results and errors, plus a workspace).  Each cluster of two CTAs
 * runs its phase-1 tiles, then its phase-2 tiles; a phase-2 tile of a unit of
 * blocks starts as soon as every phase-1 tile of that unit has stored its
 * up_logits rows (per-unit counters in `workspace`, zeroed by this call with a
 * cudaMemsetAsync on `stream`), so the phase-1 tail and the kernel boundary
 * overlap phase-2 work.  The waits are bounded (MOE_DEV_TIMEOUT) and need all
 * clusters of the launch resident at once, which the grid size ensures when
 * no other kernel holds SMs for long.  Workspace: device memory of
 * moe_single_launch_workspace_bytes(num_blocks_m) bytes, caller-owned; calls
 * that overlap on the GPU must not share it. */
moe_status_t moe_fused_forward_single_launch(
    const uint16_t* stacked_expert_tokens, int64_t total_padded_tokens, int32_t hidden,
    const uint16_t* gate_w, const uint16_t* up_w, const uint16_t* down_w,
    int32_t n_experts, int32_t intermediate,
    const float* routed_expert_weights, int64_t total_valid_tokens,
    const int32_t* group_sizes, const int32_t* group_offsets,
    const int32_t* group_padded_offsets, const int32_t* group_idx_for_bx, int64_t num_blocks_m,
    uint16_t* up_logits, uint16_t* out, void* workspace, size_t workspace_bytes,
    int32_t* status_dev, void* stream);

/* Size of the fixed workspace used by moe_fused_forward_static_workspace. */
#define MOE_STATIC_WORKSPACE_BYTES (64u * 1024u * 1024u)

/* The fused forward for callers that cannot allocate device memory (the pages
 * have no counterpart of this call).  A plugin inside an inference runtime
 * that owns every device allocation, or a latency-critical serving loop that
 * cannot afford cudaMalloc's possible device-wide synchronisation or its
 * failure under memory pressure, cannot provide the up_logits workspace that
 * moe_fused_forward needs.  This call takes the same arguments without
 * up_logits and keeps that workspace in a fixed array compiled into the
 * library: every GPU that loads the library holds MOE_STATIC_WORKSPACE_BYTES
 * (64 MiB) of device memory for it until the process exits.
 *   - Limit: total_padded_tokens * intermediate * 2 bytes must not exceed
 *     MOE_STATIC_WORKSPACE_BYTES; larger problems return
 *     MOE_ERR_STATIC_WORKSPACE and nothing is enqueued.
 *   - Allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 *   - The first call on a device looks up the array's device address with
 *     cudaGetSymbolAddress (with that device current) and caches it; make that
 *     first call before any stream capture.  The cache does not survive a
 *     device reset: do not use this call across cudaDeviceReset.
 *   - Argument checks: first the ones moe_fused_forward makes (same codes,
 *     same order), then the workspace limit (MOE_ERR_STATIC_WORKSPACE).
 *   - All calls in the process share the one array per device and it keeps
 *     the last call's contents.  Nothing in it has to start at zero.  Calls
 *     whose kernels overlap on the GPU (different streams, no ordering between
 *     them) race on the array and give wrong results; order them.
 * Otherwise the same arguments, requirements, results and errors as
 * moe_fused_forward. */
moe_status_t moe_fused_forward_static_workspace(
    const uint16_t* stacked_expert_tokens, int64_t total_padded_tokens, int32_t hidden,
    const uint16_t* gate_w, const uint16_t* up_w, const uint16_t* down_w,
    int32_t n_experts, int32_t intermediate,
    const float* routed_expert_weights, int64_t total_valid_tokens,
    const int32_t* group_sizes, const int32_t* group_offsets,
    const int32_t* group_padded_offsets, const int32_t* group_idx_for_bx, int64_t num_blocks_m,
    uint16_t* out, int32_t* status_dev, void* stream);

/* ---------------------------------------------------------------------------
 * Dense gated feed-forward block: the shared expert that every token passes
 * beside its routed experts, and the dense layers, with gradients.
 *
 * One 16-bit type for all arrays of a call (`dtype`: MOE_DTYPE_F16 or
 * MOE_DTYPE_BF16; bf16 data is passed as uint16_t bit patterns too).  Sums are
 * fp32.  hidden and intermediate are multiples of 8 (16-byte rows), at most
 * MOE_FFN_MAX_WIDTH; n_tokens is any number from 0 to MOE_FFN_MAX_TOKENS.
 * Arrays are row-major and contiguous, 16-byte aligned, and must not overlap
 * unless both are only read.
 * ------------------------------------------------------------------------- */
#define MOE_DTYPE_F16  0
#define MOE_DTYPE_BF16 1
#define MOE_DTYPE_F32  2

#define MOE_FFN_MAX_TOKENS (1 << 24)
#define MOE_FFN_MAX_WIDTH  (1 << 20)

/* Forward:
 *     G = x·gate_wᵀ, U = x·up_wᵀ           fp32
 *     up_logits = round16( G·sigmoid(G) ⊙ U )
 *     out       = round16( up_logits·down_wᵀ )
 *   x                [n_tokens, hidden]
 *   gate_w, up_w     [intermediate, hidden]
 *   down_w           [hidden, intermediate]
 *   gate, up         out, both or neither (NULL): [n_tokens, intermediate],
 *                    round16(G) and round16(U), what the backward reads
 *   up_logits        out: [n_tokens, intermediate] (workspace of a forward alone)
 *   out              out: [n_tokens, hidden]
 * Two kernel launches (the second with programmatic dependent launch).  Every
 * wait inside is bounded (2 s); one that runs out sets MOE_DEV_TIMEOUT in
 * status_dev (nullable) and leaves the outputs invalid. */
moe_status_t moe_ffn_forward(int32_t dtype, const uint16_t* x, int64_t n_tokens, int32_t hidden,
                             const uint16_t* gate_w, const uint16_t* up_w, const uint16_t* down_w,
                             int32_t intermediate, uint16_t* gate, uint16_t* up, uint16_t* up_logits,
                             uint16_t* out, int32_t* status_dev, void* stream);

/* Workspace bytes of moe_ffn_backward (the gradients of G and U, 16-bit).
 * Returns -1 for negative arguments. */
int64_t moe_ffn_backward_workspace_bytes(int64_t n_tokens, int32_t intermediate);

/* Gradients of the forward, from what it stored (gate, up, up_logits), with
 * s = sigmoid(G) and d_h = d_out·down_w in fp32:
 *     d_G = round16( d_h ⊙ U·s·(1 + G·(1 − s)) ),  d_U = round16( d_h ⊙ G·s )
 *     d_x      = round16( d_G·gate_w + d_U·up_w )    [n_tokens, hidden]
 *     d_gate_w = round16( d_Gᵀ·x )                   [intermediate, hidden]
 *     d_up_w   = round16( d_Uᵀ·x )                   [intermediate, hidden]
 *     d_down_w = round16( d_outᵀ·up_logits )         [hidden, intermediate]
 * The weights' gradients are written, not added to (zeros for n_tokens == 0).
 * workspace: device memory of moe_ffn_backward_workspace_bytes() bytes,
 * caller-owned; calls that overlap on the GPU must not share it.  Two kernel
 * launches; waits and status_dev as in the forward. */
moe_status_t moe_ffn_backward(int32_t dtype, const uint16_t* d_out, const uint16_t* x, int64_t n_tokens,
                              int32_t hidden, const uint16_t* gate_w, const uint16_t* up_w,
                              const uint16_t* down_w, int32_t intermediate, const uint16_t* gate,
                              const uint16_t* up, const uint16_t* up_logits, void* workspace,
                              size_t workspace_bytes, uint16_t* d_x, uint16_t* d_gate_w, uint16_t* d_up_w,
                              uint16_t* d_down_w, int32_t* status_dev, void* stream);

/* ---------------------------------------------------------------------------
 * 4-bit microscaled values (e2m1 codes, an e8m0 scale per 32 values of a row;
 * OCP Microscaling Formats 1.0) and products of them.
 *
 * An array of [rows, cols] values, cols a multiple of 128, is held as
 *   codes   [rows, cols/2] bytes, column 2i in the low half of byte i.  A code
 *           is sign (8) and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (0..7).
 *   scales  one byte s per 32 columns, 2^(s-127), 255 = NaN, in tiles of 128 rows
 *           x 4 blocks: [ceil(rows/128), cols/128, 32, 4, 4] with the byte of
 *           row r, block b at [r/128, b/4, r%32, r/32%4, b%4] (the order in which
 *           the tensor cores take them).
 * A weight stack [n_experts, n, k] is an array of n_experts*n rows.  Pointers are
 * 16-byte aligned; at most MOE_MX4_MAX_ROWS rows and MOE_MX4_MAX_COLS columns.
 * ------------------------------------------------------------------------- */
#define MOE_MX4_MAX_ROWS (1 << 24)
#define MOE_MX4_MAX_COLS (1 << 17)

/* Bytes of the scale tiles of [rows, cols]; -1 for arguments out of range. */
int64_t moe_mx4_scale_bytes(int64_t rows, int32_t cols);

/* Conversion to 4 bits.  With a = max |x| of a block of 32 and
 * e = max(floor(log2 a) - 2, -127), the scale byte is e + 127 and a code is
 * x·2^-e rounded to nearest even, saturated at ±6.  A block of zeros has scale
 * byte 0; a block with an infinity or NaN has scale byte 255 and codes 0.
 *   x          [n_src_rows, cols], `dtype` MOE_DTYPE_F16, _BF16 or _F32
 *   src_rows   nullable: [n_rows] int32, the rows of x to convert (otherwise
 *              n_rows must be n_src_rows); negative entries are skipped
 *   dest_rows  nullable: [n_rows, copies] int32, the row(s) of the result that
 *              each converted row goes to; negative entries are skipped, and no
 *              row may be named twice.  Otherwise copies must be 1 and row i of
 *              the list goes to row i, n_dest_rows must be n_rows, and scales
 *              past the last row of the last tile are written as 0.
 *   codes, scales  out: [n_dest_rows, cols] in 4 bits.  With dest_rows, rows not
 *              named are left as they are.
 * Entries at or past n_src_rows / n_dest_rows are skipped and set
 * MOE_DEV_BAD_TABLE.  With dest_rows = moe_pack_routed's pair_padded_rows and
 * copies = top_k this places quantised tokens in the grouped, padded layout.
 * One kernel launch. */
moe_status_t moe_mx4_quantize(int32_t dtype, const void* x, int64_t n_src_rows, int32_t cols,
                              const int32_t* src_rows, int64_t n_rows, const int32_t* dest_rows, int32_t copies,
                              int64_t n_dest_rows, uint8_t* codes, uint8_t* scales, int32_t* status_dev,
                              void* stream);

/* The values that codes and scales stand for, rounded to nearest even in
 * `dtype` where that cannot hold them: out [rows, cols].  One kernel launch. */
moe_status_t moe_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols,
                                int32_t dtype, void* out, void* stream);

/* Products of 4-bit operands with fp32 sums, on the block-scaled tensor cores;
 * results are fp16 or bf16 (`dtype`).  k, n, hidden and intermediate are
 * multiples of 128.  One kernel launch each; waits inside are bounded (2 s) as in
 * the other products (MOE_DEV_TIMEOUT).  A NaN scale of a row of A reaches only
 * that row's results.
 *
 * moe_mx4_matmul: out[i, j] = Σ_k a[i, k]·b[j, k]; a [rows, k], b [n, k], any
 * number of rows up to 128 * MOE_MAX_BLOCKS. */
moe_status_t moe_mx4_matmul(const uint8_t* a, const uint8_t* a_scales, int64_t rows, int32_t k, const uint8_t* b,
                            const uint8_t* b_scales, int32_t n, int32_t dtype, uint16_t* out,
                            int32_t* status_dev, void* stream);

/* moe_mx4_gate_up: the first half of the routed experts with 4-bit operands, in
 * the layout and with the tables of moe_fused_forward: for valid rows
 *     up_logits[p, :] = round16( silu(x[p]·gate[e]ᵀ) ⊙ (x[p]·up[e]ᵀ) )
 * x [total_padded_tokens, hidden]; gate, up [n_experts, intermediate, hidden];
 * up_logits [total_padded_tokens, intermediate], padding rows not written. */
moe_status_t moe_mx4_gate_up(const uint8_t* x, const uint8_t* x_scales, int64_t total_padded_tokens,
                             int32_t hidden, const uint8_t* gate, const uint8_t* gate_scales, const uint8_t* up,
                             const uint8_t* up_scales, int32_t n_experts, int32_t intermediate,
                             const int32_t* group_sizes, const int32_t* group_padded_offsets,
                             const int32_t* group_idx_for_bx, int64_t num_blocks_m, int32_t dtype,
                             uint16_t* up_logits, int32_t* status_dev, void* stream);

/* moe_mx4_down: the second half,
 *     out[p, :] = round16( (h[p]·down[e]ᵀ) · routed_expert_weights[c] )
 * h [total_padded_tokens, intermediate] (up_logits after moe_mx4_quantize), down
 * [n_experts, hidden, intermediate], c the row's compact index as in
 * moe_fused_forward; out [total_padded_tokens, hidden], padding rows not
 * written. */
moe_status_t moe_mx4_down(const uint8_t* h, const uint8_t* h_scales, int64_t total_padded_tokens,
                          int32_t intermediate, const uint8_t* down, const uint8_t* down_scales,
                          int32_t n_experts, int32_t hidden, const float* routed_expert_weights,
                          int64_t total_valid_tokens, const int32_t* group_sizes, const int32_t* group_offsets,
                          const int32_t* group_padded_offsets, const int32_t* group_idx_for_bx,
                          int64_t num_blocks_m, int32_t dtype, uint16_t* out, int32_t* status_dev, void* stream);

/* ---------------------------------------------------------------------------
 * Training of a routed layer: the router's losses with its per-expert counts, the
 * router's gradients, and orthogonalised updates of weight matrices.
 *
 * Tokens may be packed sequences: seq_offsets [n_seqs + 1] int32, not decreasing, in
 * [0, n_tokens]; sequence s holds tokens seq_offsets[s] .. seq_offsets[s + 1] - 1.  NULL with
 * n_seqs = 1: all tokens are one sequence.  token_mask [n_tokens] bytes, nullable: tokens with
 * 0 do not count.  A token that is masked or in no sequence enters no sum and gets a
 * gradient of zero (d_x where router_w is finite: it is zero times that), and its logits, ids, routed weights and x are
 * not used whatever they hold.  Below, T is the number of tokens that count, T_s that of sequence s, k = top_k,
 * E = n_experts, z the logits, p = softmax(z); a logit of -infinity has p = 0, and a token with
 * no other (p = 0 everywhere) adds nothing but its T and its ids.  Offsets that decrease or leave the range
 * set MOE_DEV_BAD_TABLE (in every call that has tokens) and leave the outputs undefined.  No output overlaps an input, another output or the
 * workspace.  Negative ids (moe_router_topk's for a token with too few
 * ranked logits) are skipped, ids >= n_experts too, which set MOE_DEV_BAD_EXPERT_ID.
 * ------------------------------------------------------------------------- */
#define MOE_TRAIN_MAX_TOKENS (1 << 24)
#define MOE_TRAIN_MAX_SEQS   65535

/* Workspace bytes of moe_router_balance (0 for few tokens and sequences, which need none); -1
 * for arguments out of range. */
int64_t moe_router_balance_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t n_seqs);

/* Balance loss, z loss and per-expert counts:
 *     counts[s, e] = pairs (t, j) of sequence s with id e
 *     losses[0]    = E / (k·T) · Σ_s 1/T_s · Σ_e counts[s, e] · Σ_t∈s p[t, e]
 *     losses[1]    = 1/T · Σ_t logsumexp(z[t])²
 * With one sequence losses[0] is E·Σ_e f_e·P_e, f_e the share of pairs and P_e the mean
 * probability of expert e; with several, the mean of theirs weighted by T_s.  Both are 0 where T is.
 * losses[1] is infinite where the sum of squares leaves fp32 (a row of the type's lowest value, say).
 *   logits      [n_tokens, n_experts] fp32 (moe_router_topk_logits'), 16-byte aligned
 *   topk_ids    [n_tokens, top_k] int32
 *   losses      out: [2] fp32
 *   counts      out: [n_seqs, n_experts] int32
 *   seq_tokens  out: [n_seqs + 1] int32, T_s of each sequence, then T
 *   workspace   device memory of moe_router_balance_workspace_bytes() bytes, 16-byte aligned, caller-owned;
 *               calls that overlap on the GPU must not share it
 * Limits: n_experts <= MOE_MAX_EXPERTS, top_k <= min(n_experts, MOE_ROUTER_MAX_TOPK).
 * Sums over tokens are taken in an order that does not change between calls.  One or two kernel launches. */
moe_status_t moe_router_balance(const float* logits, const int32_t* topk_ids, int64_t n_tokens, int32_t n_experts,
                                int32_t top_k, const uint8_t* token_mask, const int32_t* seq_offsets, int32_t n_seqs,
                                float* losses, int32_t* counts, int32_t* seq_tokens, void* workspace,
                                size_t workspace_bytes, int32_t* status_dev, void* stream);

/* Workspace bytes of moe_router_backward; -1 for arguments out of range. */
int64_t moe_router_backward_workspace_bytes(int64_t n_tokens, int32_t n_experts, int32_t hidden);

/* Gradients of the router, from those of the routed weights w[t, j] = p[t, id[t, j]] and of
 * the two losses (in which the counts are constants):
 *     g[t, e] = d_losses[0]·E / (k·T·T_s)·counts[s, e] + Σ_j [id[t, j] = e]·d_topk_weights[t, j]
 *     d_z     = p ⊙ (g − Σ_e p·g) + d_losses[1]·2/T·logsumexp(z)·p            fp32
 *     d_x        = round16( round16(d_z)·router_w )     [n_tokens, hidden]
 *     d_router_w = round16( round16(d_z)ᵀ·x )           [n_experts, hidden]
 * All 16-bit arrays are of `dtype` (MOE_DTYPE_F16 or _BF16).  (In fp16 d_z is rounded times a
 * power of two that depends on its largest finite magnitude, so only what is below 2^-38 of that is lost to fp16's
 * range; up to 2048 tokens, where a rounding of d_z would not average out, it is not rounded but held in two terms.)
 *   x_tokens        [n_tokens, hidden], hidden a multiple of 8, at most MOE_FFN_MAX_WIDTH
 *   router_w        [n_experts, hidden]
 *   logits, topk_ids as in moe_router_balance
 *   d_topk_weights  nullable: [n_tokens, top_k] fp32
 *   d_losses        nullable: [2] fp32, in device memory; then counts and seq_tokens of
 *                   moe_router_balance on the same tokens are needed
 *   d_x, d_router_w out, written, not added to (d_router_w zeros for n_tokens == 0)
 *   d_logits        out, nullable: d_z, [n_tokens, n_experts] fp32
 *   workspace       device memory of moe_router_backward_workspace_bytes() bytes, caller-owned;
 *                   calls that overlap on the GPU must not share it
 * x_tokens, router_w, logits, d_x, d_router_w, d_logits and workspace are 16-byte aligned.
 * Limits as in moe_router_balance.  Two to four kernel launches; waits and status_dev as in the
 * feed-forward block. */
moe_status_t moe_router_backward(int32_t dtype, const uint16_t* x_tokens, int64_t n_tokens, int32_t hidden,
                                 const uint16_t* router_w, int32_t n_experts, const float* logits,
                                 const int32_t* topk_ids, int32_t top_k, const float* d_topk_weights,
                                 const float* d_losses, const int32_t* counts, const int32_t* seq_tokens,
                                 const uint8_t* token_mask, const int32_t* seq_offsets, int32_t n_seqs, void* workspace,
                                 size_t workspace_bytes, uint16_t* d_x, uint16_t* d_router_w, float* d_logits,
                                 int32_t* status_dev, void* stream);

#define MOE_ORTHO_MAX_SIZE  (1 << 16)
#define MOE_ORTHO_MAX_BATCH 65535
#define MOE_ORTHO_MAX_STEPS 64
#define MOE_ORTHO_MAX_COEFFICIENT 64.0f

/* Workspace bytes of moe_orthogonalize; -1 for arguments out of range. */
int64_t moe_orthogonalize_workspace_bytes(int64_t batch, int32_t rows, int32_t cols);

/* Orthogonalised update: for each matrix G of the stack
 *     X = G / max(‖G‖, eps)                     (Frobenius norm)
 *     X ← a·X + (b·A + c·A²)·X, A = X·Xᵀ        `steps` times
 *     out = round16( X )                        bf16
 * which brings the singular values of G near 1 and keeps its singular vectors (a, b, c =
 * 3.4445, -4.775, 2.0315 in five steps: into about 0.7 .. 1.2 from 0.01 of the norm on).
 *   update  [batch, rows, cols], `dtype` MOE_DTYPE_F16, _BF16 or _F32
 *   out     out: [batch, rows, cols] bf16
 * Any rows and cols.  update, out and workspace are 16-byte aligned (a matrix inside a stack of odd sizes is not always).
 * Products are of fp16 operands with fp32 sums: with such coefficients the result is
 * within 2e-3 to 3e-3 of the exact one (root mean square, relative to that of the exact one, rounding to
 * bf16 included) whatever G's spectrum, so no finer type is offered; where ‖G‖ is far below eps and the result nearly
 * zero, an absolute 3e-7 besides (fp16's steps).  A matrix that holds an infinity or
 * a NaN, or whose norm leaves fp32's squares (1.8e19), becomes NaN; one of zeros stays zeros, whatever
 * eps is (0 too); the others of the stack do not see it.  The norm is taken as at least
 * 2^-69·√(rows·cols), that of entries of 1.7e-21, below which fp32's squares do not give it.  Coefficients are at most MOE_ORTHO_MAX_COEFFICIENT in magnitude, |b| at most 2048 |c|
 * unless c is 0; where they let a norm grow past 2^9 the result overflows.
 * batch·steps·ceil(rows/128)·ceil(cols/128) is at most 2^29.
 * workspace: device memory of moe_orthogonalize_workspace_bytes() bytes, caller-owned;
 * calls that overlap on the GPU must not share it.  Three kernel launches; waits and
 * status_dev as in the feed-forward block. */
moe_status_t moe_orthogonalize(int32_t dtype, const void* update, int64_t batch, int32_t rows, int32_t cols, int32_t steps,
                               float a, float b, float c, float eps, void* workspace, size_t workspace_bytes,
                               uint16_t* out, int32_t* status_dev, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
