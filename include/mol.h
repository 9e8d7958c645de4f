/*
 * mol.h - C ABI of the multi-LoRA MoE ("MoL", virtual experts) delta path on MI355X.
 *
 * One MoE layer with S LoRA adapters loaded into slots treats every (routed expert e,
 * slot l) combination as a "virtual expert" v = e + l*E, V = E*S of them. A layer pass is
 *   1. remap  - top-k base ids -> virtual ids (mol_virtual_topk, or inline in 2);
 *   2. align  - bucket the (token, slot) pairs by virtual expert into BLOCK_M-padded
 *               blocks (mol_align_block_size);
 *   3. delta  - per stage, shrink s = x A_v^T (hidden -> rank) and expand
 *               out += scale * s B_v^T (rank -> N) over the aligned blocks
 *               (mol_lora_shrink + mol_lora_expand, or fused: mol_lora_delta);
 *   4. combine - per token, the router-weighted sum of its down-stage rows
 *               (mol_moe_combine, or fused with the down expand: mol_lora_expand_combine).
 * Sources: the sglang virtual-experts kernels as summarised on the PR 24171 page
 * (remap keeping negative sentinels, sentinel bucket, -1 blocks skipped), the PR 24262
 * page (align as histogram -> prefix sum -> expert ids -> scatter, no host sync, the
 * 8192-bucket ceiling), and MindLab sglang PR 24 (shrink/expand stage shapes, weights
 * laid out [E, N, K] with N = shape[1], the "-1 = no adapter" slot contract).
 *
 * Conventions for every entry point:
 *  - Pointers are DEVICE pointers unless marked (host). The caller owns every buffer,
 *    including workspaces; the library keeps no device memory of its own.
 *  - Calls only validate host-side scalars and pointers, then enqueue kernels on
 *    `stream` (a hipStream_t; NULL = the legacy default stream) and return. No call
 *    allocates, synchronises, or reads device memory on the host, so a sequence of calls
 *    can be captured into a hipGraph.
 *  - Bad *device data* cannot be reported without a sync; it has defined behaviour
 *    instead: a base id >= E, a slot outside [0, S) and any negative id never reach a
 *    real virtual expert (they land in the sentinel bucket and get no delta).
 *  - Matrices are row-major; "ld" arguments are row strides in elements.
 *  - Returns MOL_OK or an error code; nothing is enqueued when an error is returned
 *    (except MOL_E_HIP, which reports a failed launch).
 */
#ifndef MOL_H
#define MOL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define MOL_API __attribute__((visibility("default")))
#else
#define MOL_API
#endif

typedef int32_t mol_status;

enum {
    MOL_OK = 0,
    MOL_E_ARG = 1,       /* NULL pointer, negative or zero size, inconsistent shapes   */
    MOL_E_LIMIT = 2,     /* more than MOL_MAX_BUCKETS buckets, rank or block too large */
    MOL_E_DTYPE = 3,     /* unknown dtype                                              */
    MOL_E_ALIGN = 4,     /* a row, stride or base pointer not 16-byte aligned          */
    MOL_E_WORKSPACE = 5, /* workspace missing or smaller than the size query says      */
    MOL_E_HIP = 6        /* a HIP call or kernel launch failed                         */
};

enum { MOL_F32 = 0, MOL_BF16 = 1 };

/* At most 8192 buckets = 8191 virtual experts + the sentinel bucket (the align kernel
 * ceiling on the PR 24262 page). */
#define MOL_MAX_BUCKETS 8192
#define MOL_MAX_BLOCK_M 1024
/* expand: r * sizeof(elem) <= 256 bytes (rank <= 128 in bf16, <= 64 in fp32) */
#define MOL_MAX_RANK_BYTES 256
/* floats of the library's own per-GPU scratch behind mol_lora_delta_noalloc (16 MiB) */
#define MOL_DELTA_SCRATCH_FLOATS (4 * 1024 * 1024)

/* (host) Static description of a status code. Never NULL. */
MOL_API const char *mol_status_string(mol_status status);

/* (host) ABI version of this header, 7 (2 added the per-slot ranks, 3 the combine, 4 the
 * base grouped GEMM with the fused delta, 5 the allocation-free stage delta, 6 the work
 * plan, 7 the plan as runs of blocks only, read by the expand). Entry points that leave the
 * earlier ones as they are (mol_router_topk and those after it) come within a version. */
MOL_API int32_t mol_abi_version(void);

/* ---------------------------------------------------------------------------------
 * mol_virtual_topk - remap base top-k ids to virtual ids (PR 24171 page: the fused
 * virtual top-k ids kernel keeps a negative id and shifts the others by slot * E).
 *   topk_ids     int32 [M, topk]   base expert ids; negative = expert-parallel sentinel
 *   lora_ids     int32 [M]         LoRA slot per token; -1 = no adapter
 *   virtual_ids  int32 [M, topk]   out: t if t < 0; -1 if t >= E or slot outside [0, S);
 *                                  else t + slot * E. May not alias the inputs.
 * M == 0 is valid and enqueues nothing. Errors: MOL_E_ARG.
 * ------------------------------------------------------------------------------- */
MOL_API mol_status mol_virtual_topk(const int32_t *topk_ids, const int32_t *lora_ids,
                                    int32_t M, int32_t topk, int32_t num_experts,
                                    int32_t num_slots, int32_t *virtual_ids, void *stream);

/* ---------------------------------------------------------------------------------
 * Align sizing (host, pure). num_virtual = V = E * S.
 *   mol_align_max_blocks: an upper bound on the number of BLOCK_M blocks any routing
 *     of `numel` pairs can produce, cdiv(numel + min(numel, V+1) * (block_m - 1),
 *     block_m). sorted_ids needs max_blocks * block_m entries, expert_ids max_blocks.
 *   mol_align_workspace_bytes: device workspace mol_align_block_size needs (0 when the
 *     one-workgroup kernel handles numel).
 * Both return a negative -mol_status on invalid arguments (e.g. -MOL_E_LIMIT when
 * V + 1 > MOL_MAX_BUCKETS).
 * ------------------------------------------------------------------------------- */
MOL_API int64_t mol_align_max_blocks(int64_t numel, int32_t num_virtual, int32_t block_m);
MOL_API int64_t mol_align_workspace_bytes(int64_t numel, int32_t num_virtual, int32_t block_m);

/* ---------------------------------------------------------------------------------
 * The work plan (optional). A batch of at least 4096 pairs and 8 pairs per bucket on average
 * (numel >= 8 (V + 1)) is dense enough for the bf16 matrix-core kernels, which then take
 * every block (no VALU kernel is launched). For such a batch, mol_align_block_size can write
 * beside the routing a plan of its blocks: runs of up to four consecutive blocks of one
 * virtual expert, every block of a real bucket in exactly one run. The expand then takes
 * whole runs as work items and loads each weight column once per run instead of once per
 * block. For other batches nothing is written and the calls ignore a plan. Layout (int32
 * words): [0] the number of runs, [1..7] 0; from word 8, runs of 4 words {first block,
 * blocks (1..4), virtual expert, 0} in bucket order, at most min(max_blocks, numel). The
 * sentinel bucket has none.
 *   mol_plan_bytes: bytes of a plan buffer (a multiple of 256), or -mol_status.
 * ------------------------------------------------------------------------------- */
MOL_API int64_t mol_plan_bytes(int64_t numel, int32_t num_virtual, int32_t block_m);

/* ---------------------------------------------------------------------------------
 * mol_align_block_size - bucket the numel = M * topk pairs by virtual expert (PR 24262
 * page: histogram, padded prefix sum, per-block expert ids, token scatter; PR 24171
 * page: the extra sentinel bucket whose blocks are -1).
 *   ids            int32 [M, topk]  base ids (lora_ids != NULL: remapped inline exactly
 *                                   as mol_virtual_topk) or virtual ids (lora_ids == NULL)
 *   lora_ids       int32 [M] or NULL
 *   Bucket of a pair = its virtual id if in [0, V), else V (the sentinel bucket, last).
 *   With c_b pairs in bucket b, pc_b = ceil(c_b / block_m) * block_m and off_b the
 *   exclusive prefix sum of pc:
 *   sorted_ids       int32 [max_blocks * block_m] out: sorted_ids[off_b + j] = the j-th
 *                    pair of bucket b in ascending pair order (j < c_b); entries
 *                    [off_b + c_b, off_b + pc_b) = numel (padding).
 *   expert_ids       int32 [max_blocks] out: block i in [off_b, off_b + pc_b)/block_m
 *                    gets b, or -1 for the sentinel bucket.
 *   num_post_padded  int32 [1] out: sum_b pc_b.
 *   Entries past num_post_padded (resp. num_post_padded / block_m) are left undefined.
 *   plan, plan_bytes the work plan out (see above; 16-byte aligned, at least
 *                    mol_plan_bytes()), or NULL (0). Written only for a batch that takes
 *                    the matrix-core kernels; the buffer is left untouched otherwise.
 *   workspace        device scratch of mol_align_workspace_bytes(), or NULL when that is 0.
 * No atomics are used; results are bit-for-bit reproducible. M == 0 writes
 * num_post_padded = 0 (sorted_ids and expert_ids may then be NULL).
 * Errors: MOL_E_ARG, MOL_E_LIMIT (V + 1 > MOL_MAX_BUCKETS, block_m > MOL_MAX_BLOCK_M),
 * MOL_E_WORKSPACE, MOL_E_HIP.
 * ------------------------------------------------------------------------------- */
MOL_API mol_status mol_align_block_size(const int32_t *ids, const int32_t *lora_ids,
                                        int32_t M, int32_t topk, int32_t num_experts,
                                        int32_t num_slots, int32_t block_m,
                                        int32_t *sorted_ids, int32_t *expert_ids,
                                        int32_t *num_post_padded, int32_t *plan,
                                        size_t plan_bytes, void *workspace,
                                        size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------
 * Per-slot ranks (all three delta calls). slot_ranks, int32 [num_virtual / num_experts] or
 * NULL, gives the rank rl of each LoRA slot (MindLab sglang PR 24: the lora_ranks table and
 * its rank == 0 early return): an adapter of rank rl uses rank dimensions [0, rl) of each
 * slice of its weights, r = R / slices. Values are clamped to [0, r]; NULL means every slot
 * has rank r. Weights past a slot's rank are never read, whatever they hold.
 * ------------------------------------------------------------------------------- */

/* ---------------------------------------------------------------------------------
 * mol_lora_shrink - s[p, i] = sum_k A[v, i, k] * xin[p / row_div, k] for every real pair
 * p of every block with expert id v >= 0 (MindLab sglang PR 24: the MoL shrink stage,
 * hidden -> rank). fp32 accumulation.
 *   dtype        MOL_F32 or MOL_BF16 (xin and A)
 *   xin          [rows, ld_x] input rows; pair p reads row p / row_div (row_div = topk
 *                for token rows, 1 for per-pair rows)
 *   A            [V, R, K] weights, rows of K contiguous elements
 *   slices       R = slices * r; slice g holds rank dimensions [g r, g r + r)
 *   slot_ranks, num_experts: the per-slot ranks above (slot of v = v / num_experts);
 *                s[p, g r + i] = 0 for i >= rl
 *   sorted_ids, expert_ids, num_post_padded: the outputs of mol_align_block_size for
 *                `numel` pairs, V = num_virtual virtual experts and this block_m
 *   s            float32 [numel, R] out, 16-byte aligned; rows of pairs that get no delta are
 *                untouched
 * Requires K * elem and ld_x * elem to be multiples of 16 bytes, R % slices == 0, and xin,
 * A, s 16-byte aligned (MOL_E_ALIGN). numel == 0 enqueues nothing.
 * ------------------------------------------------------------------------------- */
MOL_API mol_status mol_lora_shrink(int32_t dtype, const void *xin, int64_t ld_x,
                                   int32_t row_div, const void *A, int32_t R, int32_t K,
                                   int32_t slices, const int32_t *slot_ranks,
                                   int32_t num_experts, const int32_t *sorted_ids,
                                   const int32_t *expert_ids, const int32_t *num_post_padded,
                                   int32_t numel, int32_t num_virtual, int32_t block_m,
                                   float *s, void *stream);

/* ---------------------------------------------------------------------------------
 * mol_lora_expand - for the same pairs, with r = R / slices, w = N / slices and rl the
 * slot's rank,
 *   out[p, n] = round(out[p, n] + slot_scale[v / E] * sum_{j < rl} B[v, n, j] * s[p, (n / w) * r + j])
 * (MindLab sglang PR 24: expand rank -> N; gate_up expands as two slices, gate from
 * s[:, :r] and up from s[:, r:]). Sum in fp32, one fused multiply-add into the fp32 value
 * of out, then round to nearest even for bf16. A slot of rank 0 adds nothing.
 *   s            float32 [numel, R] from mol_lora_shrink, 16-byte aligned
 *   B            [V, N, r] weights (dtype as out)
 *   slot_scale   float32 [num_virtual / num_experts]
 *   slot_ranks   int32 [num_virtual / num_experts] or NULL (see above)
 *   out          [numel, ld_out] read and written in place; rows of pairs without a
 *                delta are left bit-for-bit untouched
 *   plan         the work plan the same align call wrote, or NULL. When the matrix-core
 *                kernels take the batch, their items are then the plan's runs (same
 *                results); otherwise it is not read. (mol_lora_delta and
 *                mol_lora_delta_noalloc take the same argument for their expand.)
 * Requires R % slices == 0, N % slices == 0, r * elem a multiple of 16 bytes and at most
 * MOL_MAX_RANK_BYTES, B and s 16-byte aligned (MOL_E_ALIGN), out aligned to its element.
 * ------------------------------------------------------------------------------- */
MOL_API mol_status mol_lora_expand(int32_t dtype, const float *s, int32_t R, int32_t slices,
                                   const void *B, int32_t N, const float *slot_scale,
                                   const int32_t *slot_ranks, int32_t num_experts,
                                   const int32_t *sorted_ids, const int32_t *expert_ids,
                                   const int32_t *num_post_padded, const int32_t *plan,
                                   int32_t numel, int32_t num_virtual, int32_t block_m,
                                   void *out, int64_t ld_out, void *stream);

/* ---------------------------------------------------------------------------------
 * mol_lora_delta - one stage: shrink then expand, with s kept in the caller's workspace.
 * Same arguments and results as mol_lora_shrink followed by mol_lora_expand (bit-identical
 * to them; they are the same kernels, enqueued back to back).
 *   workspace    device scratch of at least mol_delta_workspace_bytes(), 16-byte aligned;
 *                no initial contents are required. Calls that may overlap must not share
 *                a workspace.
 * ------------------------------------------------------------------------------- */
MOL_API int64_t mol_delta_workspace_bytes(int32_t numel, int32_t R, int32_t num_virtual,
                                          int32_t block_m);
MOL_API mol_status mol_lora_delta(int32_t dtype, const void *xin, int64_t ld_x,
                                  int32_t row_div, const void *A, int32_t R, int32_t K,
                                  int32_t slices, const void *B, int32_t N,
                                  const float *slot_scale, const int32_t *slot_ranks,
                                  int32_t num_experts, const int32_t *sorted_ids,
                                  const int32_t *expert_ids, const int32_t *num_post_padded,
                                  const int32_t *plan, int32_t numel, int32_t num_virtual,
                                  int32_t block_m, void *out, int64_t ld_out, void *workspace,
                                  size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------
 * mol_lora_delta_noalloc - mol_lora_delta for callers that cannot allocate device memory
 * (code under hipGraph capture, tight serving loops, harnesses that forbid hipMalloc): the
 * same checks, kernels and results (bit-identical), but s lives in a scratch array that the
 * library itself holds on each GPU, so no workspace is passed and nothing is allocated.
 *   Limit: numel * R <= MOL_DELTA_SCRATCH_FLOATS (16 MiB of float32), else MOL_E_LIMIT
 *          before anything is enqueued. The scratch needs no initial contents.
 *   Every call on one GPU shares that GPU's scratch and leaves its contents behind: calls
 *   that may overlap on one GPU (other streams, other threads) race and must not be made.
 *   The first call on a device looks up the scratch's address there (no allocation); a
 *   failure of that lookup returns MOL_E_HIP. Other errors as for mol_lora_delta.
 * ------------------------------------------------------------------------------- */
MOL_API mol_status mol_lora_delta_noalloc(int32_t dtype, const void *xin, int64_t ld_x,
                                          int32_t row_div, const void *A, int32_t R,
                                          int32_t K, int32_t slices, const void *B, int32_t N,
                                          const float *slot_scale, const int32_t *slot_ranks,
                                          int32_t num_experts, const int32_t *sorted_ids,
                                          const int32_t *expert_ids,
                                          const int32_t *num_post_padded,
                                          const int32_t *plan, int32_t numel,
                                          int32_t num_virtual, int32_t block_m, void *out,
                                          int64_t ld_out, void *stream);

/* ---------------------------------------------------------------------------------
 * mol_moe_gemm - the base MoE grouped GEMM of a stage, with the LoRA delta optionally fused
 * into its epilogue. The pages' layer runs the base grouped-GEMM launches and then the LoRA
 * launches that add the delta into the same rows (MindLab sglang PR 24, the PR body's count
 * of base and LoRA launches per layer); fused, the rows are written once:
 *   out[p, n] = round( sum_k W[t, n, k] * xin[p / row_div, k]
 *                      + slot_scale[l] * sum_{j < rl} B[t + l*E, n, j] * s[p, (n / w) * r + j] )
 * for every pair p with a local base expert t = topk id in [0, E) (other rows untouched),
 * with l the token's slot (lora_ids[p / topk]; the delta term only for l in [0, S) and slot
 * rank rl > 0), r = R / slices, w = N / slices. Summed in fp32, rounded once (bf16 RNE).
 *   sorted_ids, expert_ids, num_post_padded
 *                 the routing by BASE expert: mol_align_block_size over the top-k ids with
 *                 lora_ids = NULL and num_slots = 1 (num_virtual = num_experts)
 *   W             [E, N, K] base weights (dtype), 16-byte aligned, K * elem a multiple of 16
 *   xin           rows of ld_x elements (16-byte multiple), row p / row_div for pair p
 *   out           [numel, ld_out] (dtype), aligned to its element
 *   s             NULL: the base GEMM alone. Else the fused delta: float32 [numel, R] from
 *                 mol_lora_shrink of the same stage (16-byte aligned), B [E*S, N, r] (dtype,
 *                 16-byte aligned), slot_scale [S], slot_ranks [S] or NULL, lora_ids [numel /
 *                 topk]; r * elem a multiple of 16 and at most MOL_MAX_RANK_BYTES
 * Built for decode-sized batches (a gather of matrix-vector products over the touched
 * experts' weights, like the shrink). Errors as for mol_lora_shrink / mol_lora_expand.
 * ------------------------------------------------------------------------------- */
MOL_API mol_status mol_moe_gemm(int32_t dtype, const void *xin, int64_t ld_x, int32_t row_div,
                                const void *W, int32_t K, int32_t N, int32_t num_experts,
                                const int32_t *sorted_ids, const int32_t *expert_ids,
                                const int32_t *num_post_padded, int32_t numel, int32_t block_m,
                                void *out, int64_t ld_out, const float *s, int32_t R,
                                int32_t slices, const void *B, const float *slot_scale,
                                const int32_t *slot_ranks, const int32_t *lora_ids,
                                int32_t topk, int32_t num_slots, void *stream);

/* ---------------------------------------------------------------------------------
 * The combine after the down projection. The pages stop at the per-pair rows the down
 * stage's delta is added into (the layer's grouped-GEMM launches counted on the MindLab
 * sglang PR 24 page end with the down expand); the next step of an MoE layer sums each
 * token's pair rows with its router weights. A pair whose base id is outside [0, E) has no
 * local expert (a negative id is an expert-parallel sentinel: the expert lives on another
 * GPU) and contributes nothing; its row is never read.
 *
 * mol_moe_combine -
 *   y[m, n] = round( sum_{k ascending, 0 <= topk_ids[m, k] < E} w[m, k] * rows[m*topk + k, n] )
 * summed in fp32 and rounded once (bf16: to nearest even).
 *   rows          [M*topk, ld_rows] pair rows (dtype), e.g. the down stage's out
 *   topk_ids      int32 [M, topk] base expert ids
 *   topk_weights  float32 [M, topk] router weights
 *   y             [M, ld_y] out (dtype); every element of [M, N] is written
 * Requires N, ld_rows and ld_y multiples of 16 bytes' worth of elements (8 bf16, 4 fp32)
 * and rows, y 16-byte aligned (MOL_E_ALIGN). M = 0 is a no-op.
 * ------------------------------------------------------------------------------- */
MOL_API mol_status mol_moe_combine(int32_t dtype, const void *rows, int64_t ld_rows,
                                   const int32_t *topk_ids, const float *topk_weights,
                                   int32_t M, int32_t topk, int32_t num_experts, int32_t N,
                                   void *y, int64_t ld_y, void *stream);

/* ---------------------------------------------------------------------------------
 * mol_lora_expand_combine - the down stage's expand (one slice) fused with the combine;
 * the per-pair rows are never written:
 *   y[m, n] = round( sum_{k, 0 <= t < E} w[m, k] * (base[p, n] + d_p[n]) ),  p = m*topk + k,
 *   d_p[n]  = slot_scale[l] * sum_{j < rl} B[v, n, j] * s[p, j]
 * for a pair whose token has slot l in [0, S) (virtual expert v = t + l*E, slot rank rl >
 * 0); otherwise d_p = 0. Summed in fp32, rounded once. It reads each pair's B_v columns,
 * which at decode (almost every pair its own virtual expert) are the same bytes the aligned
 * expand reads; with many tokens per virtual expert (prefill) mol_lora_expand followed by
 * mol_moe_combine reads far fewer.
 *   s             float32 [M*topk, R] from mol_lora_shrink of the down stage, 16-byte
 *                 aligned; rows of pairs without a delta are not read
 *   B             [E*S, N, R] (dtype), 16-byte aligned
 *   slot_scale    float32 [S];  slot_ranks  int32 [S] or NULL (clamped to [0, R])
 *   lora_ids      int32 [M] LoRA slot per token (-1: no adapter, base row only)
 *   base          [M*topk, ld_base] the pairs' base rows (read only)
 *   y             [M, ld_y] out
 * Requires R * elem a multiple of 16 bytes with R / (16 / elem) a power of two up to 16
 * (bf16 ranks 8..128, fp32 ranks 4..64; else MOL_E_LIMIT), E*S + 1 <= MOL_MAX_BUCKETS.
 * ------------------------------------------------------------------------------- */
MOL_API mol_status mol_lora_expand_combine(int32_t dtype, const float *s, int32_t R,
                                           const void *B, int32_t N, const float *slot_scale,
                                           const int32_t *slot_ranks, const int32_t *topk_ids,
                                           const int32_t *lora_ids,
                                           const float *topk_weights, int32_t M, int32_t topk,
                                           int32_t num_experts, int32_t num_slots,
                                           const void *base, int64_t ld_base, void *y,
                                           int64_t ld_y, void *stream);

/* ---------------------------------------------------------------------------------
 * mol_router_topk - from router logits to the top-k experts of each token and their weights:
 * the topk_ids and topk_weights that the calls above take.
 *   logits        [M, ld_logits] (dtype), one row of num_experts logits per token
 *   Candidates of a row are its logits that are neither NaN nor -infinity (an expert is
 *   masked by either). Slot j gets the candidate with the j-th largest logit, equal logits in
 *   ascending expert order; slots past the last candidate get id -1 and weight 0.
 *   scoring       MOL_SCORE_SOFTMAX: score = exp(l - max) / sum over the candidates of exp(l - max)
 *                 (rows that hold +infinity share 1 among those entries);
 *                 MOL_SCORE_SIGMOID: score = 1 / (1 + exp(-l))
 *   renormalize   nonzero: each score is divided by the sum of the row's selected scores
 *   scale         finite factor on the weights, applied last
 *   first_expert, num_local
 *                 the experts this GPU holds: a selected expert e gets id e - first_expert
 *                 inside [first_expert, first_expert + num_local), else id -1 and weight 0 (the
 *                 expert-parallel sentinel of the calls above). 0 and num_experts for all.
 *                 Selection, scores and renormalization are over all num_experts.
 *   topk_ids      int32 [M, topk] out;  topk_weights  float32 [M, topk] out
 * Scores and sums are fp32. logits is aligned to its element, at any row stride >= num_experts.
 * Errors: MOL_E_ARG, MOL_E_DTYPE, MOL_E_ALIGN, MOL_E_LIMIT (num_experts + 1 > MOL_MAX_BUCKETS,
 * topk > MOL_MAX_ROUTER_TOPK, M * topk past 32 bits, more than 2^28 - 16 tokens, or 2^26 - 4 with over
 * 256 experts or 16 slots). M = 0 is a no-op.
 * ------------------------------------------------------------------------------- */
enum { MOL_SCORE_SOFTMAX = 0, MOL_SCORE_SIGMOID = 1 };
#define MOL_MAX_ROUTER_TOPK 64

MOL_API mol_status mol_router_topk(int32_t dtype, const void *logits, int64_t ld_logits,
                                   int32_t M, int32_t num_experts, int32_t topk,
                                   int32_t scoring, int32_t renormalize, float scale,
                                   int32_t first_expert, int32_t num_local, int32_t *topk_ids,
                                   float *topk_weights, void *stream);

/* ---------------------------------------------------------------------------------
 * The balance loss of a routed batch (the auxiliary loss that keeps a router's experts evenly
 * used), the experts' counts, and the gradient in the logits. A token counts if its mask is not zero
 * and its row has a candidate (a logit that is neither NaN nor -infinity, as above). Over the n tokens
 * that count, with c_e the number of their ids that are e and p_me their scores over the row's candidates
 * (MOL_SCORE_SOFTMAX: softmax; MOL_SCORE_SIGMOID: sigmoids divided by their sum):
 *   P_e  = sum_m p_me
 *   loss = alpha * E / (topk * n^2) * sum_e c_e P_e            (alpha for an even batch; 0 if n = 0)
 *   d loss / d l_mj = p_mj q_mj (a_j - sum_e p_me a_e),  a_e = alpha * E * c_e / (topk * n^2),
 *                     q = 1 (softmax) or 1 - sigmoid(l_mj); 0 for masked logits and tokens that
 *                     do not count
 * Counts are constants to the gradient, as ids are.
 *
 * mol_router_balance -
 *   logits        [M, ld_logits] (dtype), aligned to its element;  topk_ids  int32 [M, topk], the ids
 *                 chosen for the tokens over all experts (ids outside [0, E) are not counted: -1
 *                 for slots past the last candidate)
 *   token_mask    uint8 [M]: 0 for tokens that do not count (padding), or NULL
 *   alpha         finite factor of the loss
 *   counts        int32 [num_experts + 1] out: c_e, then n
 *   prob_sums     float32 [num_experts] out: P_e;   loss  float32 [1] out
 *   workspace     device scratch of mol_router_balance_workspace_bytes(), 16-byte aligned (NULL when
 *                 that is 0); needs no initial contents. Calls that may overlap must not share it.
 * Bit-for-bit reproducible: no sum depends on timing. M = 0 writes zeros. A workgroup's sums are fp32, the
 * sums over workgroups are formed in 64 bits.
 *
 * mol_router_balance_grad - grad_logits [M, ld_grad] (dtype) out, every element of [M, num_experts]:
 *   counts        int32 [num_experts + 1] of mol_router_balance, or their sums over the ranks that
 *                 share the batch (the loss is then that of the whole batch: its P_e are sums too)
 *   grad_loss     float32 [1], the gradient that arrives at the loss, or NULL for 1
 *   others        as above. grad_logits may be logits itself (with its stride). M = 0 enqueues nothing.
 * Errors of both: MOL_E_ARG, MOL_E_DTYPE, MOL_E_ALIGN, MOL_E_WORKSPACE, MOL_E_LIMIT (num_experts + 1 >
 * MOL_MAX_BUCKETS, topk > MOL_MAX_ROUTER_TOPK, M * topk past 32 bits).
 * ------------------------------------------------------------------------------- */
/* bytes of a workspace for up to M tokens, or -mol_status */
MOL_API int64_t mol_router_balance_workspace_bytes(int32_t M, int32_t num_experts);
MOL_API mol_status mol_router_balance(int32_t dtype, const void *logits, int64_t ld_logits,
                                      const int32_t *topk_ids, const uint8_t *token_mask,
                                      int32_t M, int32_t num_experts, int32_t topk,
                                      int32_t scoring, float alpha, int32_t *counts,
                                      float *prob_sums, float *loss, void *workspace,
                                      size_t workspace_bytes, void *stream);
MOL_API mol_status mol_router_balance_grad(int32_t dtype, const void *logits, int64_t ld_logits,
                                           const uint8_t *token_mask, const int32_t *counts,
                                           const float *grad_loss, int32_t M,
                                           int32_t num_experts, int32_t topk, int32_t scoring,
                                           float alpha, void *grad_logits, int64_t ld_grad,
                                           void *stream);

/* ---------------------------------------------------------------------------------
 * 4-bit weights. A matrix of N rows of K weights is stored as uint8 [N, K / 2], two per byte:
 * byte b of a row holds k = 2b in its low half and k = 2b + 1 in its high half, each an
 * unsigned q in 0..15. Every group of G (32, 64 or 128) consecutive k's of a row has a scale and
 * optionally a zero point: weight = (q - z) * scale. scales [N, K / G] has the dtype of the
 * input rows; zeros uint8 [N, K / G] holds any value 0..255, NULL means 8 throughout.
 * K is a multiple of G, of at most 256 groups.
 *
 * mol_moe_gemm_q4 - mol_moe_gemm's base product over such weights:
 *   out[p, n] = round( sum_k (q[t,n,k] - z[t,n,k/G]) * scale[t,n,k/G] * xin[p / row_div, k] )
 * for every pair p with a local base expert t in [0, E); other rows are untouched. Summed in
 * fp32, the scale applied to a group's sum, rounded once; a sum that is not finite then (an infinite
 * x, or values near the largest float) is formed again from its terms, each weight scaled first, so
 * infinities and NaN are the formula's. num_experts = 1 and ids of zero give the product with a
 * single matrix.
 *   dtype         MOL_F32 or MOL_BF16: xin, scales and out
 *   W             uint8 [E, N, K / 2], 16-byte aligned;  scales [E, N, K / group], aligned to
 *                 its element;  zeros uint8 [E, N, K / group] or NULL
 *   others        as for mol_moe_gemm (rows of xin on 16-byte boundaries)
 * Built for decode-sized batches; blocks of any block_m are taken.
 * Errors: MOL_E_ARG (a group that is not 32, 64 or 128, K not a multiple of it), MOL_E_LIMIT
 * (more than 256 groups a row, one expert's weights 2 GiB or more, 2^24 work items or more), others
 * as for mol_moe_gemm.
 * ------------------------------------------------------------------------------- */
MOL_API mol_status mol_moe_gemm_q4(int32_t dtype, const void *xin, int64_t ld_x, int32_t row_div,
                                   const uint8_t *W, const void *scales, const uint8_t *zeros,
                                   int32_t group, int32_t K, int32_t N, int32_t num_experts,
                                   const int32_t *sorted_ids, const int32_t *expert_ids,
                                   const int32_t *num_post_padded, int32_t numel,
                                   int32_t block_m, void *out, int64_t ld_out, void *stream);

/* ---------------------------------------------------------------------------------
 * Microscaled 4-bit floats (MX4). A row of K values is stored as uint8 [K / 2], two per byte: byte
 * b holds k = 2b in its low half and k = 2b + 1 in its high half, each a code of a sign bit (the
 * highest) and one of the eight magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6 in this order. Every 32 consecutive
 * values share a scale byte s of uint8 [K / 32], which stands for 2^(s - 127); s = 255 makes the 32
 * NaN. K is a multiple of 32. (The element and scale formats of the OCP Microscaling specification, MXFP4.)
 *
 * mol_mx4_quantize - rows to codes and scales. With m the largest magnitude of a block:
 *   s = max(floor(log2 m) - 2, -127) + 127;  each value over 2^(s - 127) to the nearest magnitude, halves to
 *   the even code, beyond 6 to 6. A block with a NaN or an infinity gets s = 255 and codes of zero.
 *   activation    MOL_ACT_NONE: x [rows, K], the values;  MOL_ACT_SILU_MUL: x [rows, 2 K], gate
 *                 columns first, value k = SiLU(x[k]) * x[K + k] (the rows of a layer's gate_up product,
 *                 for its down product). Its codes are those of the value in 64 bits; a value of 2^128 or
 *                 more counts as infinite.
 *   x             rows of ld_x elements (dtype), aligned to its element
 *   q             uint8 [rows, K / 2] out, 16-byte aligned;  scales  uint8 [rows, K / 32] out
 * mol_mx4_dequantize - the values of codes and scales, x [rows, ld_x] (dtype) out: exact in both dtypes
 *   up to s = 252, infinite where they pass fp32's range beyond.
 * rows = 0 enqueues nothing. Errors: MOL_E_ARG, MOL_E_DTYPE, MOL_E_ALIGN, MOL_E_LIMIT (rows * K / 8
 * past 2^30 - 4096).
 *
 * mol_moe_gemm_mx4 - mol_moe_gemm's base product over such weights:
 *   out[p, n] = round( sum_k W[t, n, k] * xin[p / row_div, k] )
 * for every pair p with a local base expert t in [0, E); other rows are untouched. Products and sums
 * are fp32, rounded once. num_experts = 1 and ids of zero give the product with a single matrix. Beside
 * bf16 or fp32 rows a weight is its value in fp32: infinite from 2^128 on (some codes at s = 253 and 254);
 * beside rows of codes any two scales multiply as powers of two.
 *   dtype         MOL_F32 or MOL_BF16 of out, and of xin without x_scales
 *   xin, x_scales x_scales NULL: rows of ld_x elements (dtype). Else rows of codes, ld_x / 2 bytes apart
 *                 (ld_x a multiple of 32), with scales ld_x / 32 bytes apart
 *   W             uint8 [E, N, K / 2], 16-byte aligned;  scales uint8 [E, N, K / 32]
 *   others        as for mol_moe_gemm (rows of xin on 16-byte boundaries)
 * For decode and prefill batches; blocks of any block_m are taken. From some thousand tokens on blocks of 128
 * pairs run fastest; of 64, 32 or 16 of one expert in a row, full but for the last, are taken together (not beside
 * fp32 rows).
 * Errors: MOL_E_ARG (K not a multiple of 32), MOL_E_LIMIT (one expert's weights 2 GiB or more; 2^32 threads
 * or more, which are 2^24 work items, 2^23 of many pairs of codes or bf16 rows), others as for mol_moe_gemm.
 * ------------------------------------------------------------------------------- */
enum { MOL_ACT_NONE = 0, MOL_ACT_SILU_MUL = 1 };

MOL_API mol_status mol_mx4_quantize(int32_t dtype, int32_t activation, const void *x,
                                    int64_t ld_x, int64_t rows, int32_t K, uint8_t *q,
                                    uint8_t *scales, void *stream);
MOL_API mol_status mol_mx4_dequantize(int32_t dtype, const uint8_t *q, const uint8_t *scales,
                                      int64_t rows, int32_t K, void *x, int64_t ld_x,
                                      void *stream);
MOL_API mol_status mol_moe_gemm_mx4(int32_t dtype, const void *xin, int64_t ld_x,
                                    const uint8_t *x_scales, int32_t row_div, const uint8_t *W,
                                    const uint8_t *scales, int32_t K, int32_t N,
                                    int32_t num_experts, const int32_t *sorted_ids,
                                    const int32_t *expert_ids, const int32_t *num_post_padded,
                                    int32_t numel, int32_t block_m, void *out, int64_t ld_out,
                                    void *stream);

/* ---------------------------------------------------------------------------------
 * mol_moe_layer - a whole layer for a few tokens, from the routed ids to the combined rows, with
 * no aligned routing: two launches for a token, or up to three of them, without adapters (gate/up
 * with the activation, down with the combine); three beyond (the combine on its own); four with
 * adapters (the activation too; their products run beside the base ones). For pair
 * p = m * topk + k with a local base expert t = topk_ids[m, k] in [0, E), and l = lora_ids[m] (the
 * adapter terms only for l in [0, S) and slot rank rl > 0, v = t + l * E):
 *   g    = gate_up[t, 0:I] x_m + slot_scale[l] * gate_up_B[v, 0:I, :rl] (gate_up_A[v, 0:rl] x_m)
 *   u    = gate_up[t, I:2I] x_m + slot_scale[l] * gate_up_B[v, I:2I, :rl] (gate_up_A[v, r:r+rl] x_m)
 *   h_p  = g / (1 + exp(-g)) * u
 *   y_m  = round( sum_k topk_weights[m, k] * (down[t] h_p
 *                  + slot_scale[l] * down_B[v, :, :rl] (down_A[v, 0:rl] h_p)) )
 * Pairs without a local expert contribute nothing; a token that has none gets a row of
 * zeros. Sums, g, u and h are fp32 (SiLU within 2^-20 of itself); bf16 products take h, and
 * the adapters' products A x and A h where B multiplies them, as two bf16 terms each (at least 16 of
 * their bits); y alone is rounded to bf16 (to nearest even). Sums over 4-bit weights and over two terms
 * that are not finite are formed again from their terms: infinities and NaN are the formula's.
 *   w             (host) the weights; read during the call only. dtype: MOL_F32 or MOL_BF16 of x,
 *                 y, the scales, the adapters, and of the weights themselves when group is 0.
 *                 gate_up [E, 2 * inter, hidden] (gate rows first), down [E, hidden, inter],
 *                 16-byte aligned. group 32, 64 or 128: 4-bit weights (above) with their
 *                 scales and zero points (zeros may be NULL); group 0: no scales, no zeros.
 *   adapters      (host) the adapters of S = num_slots slots, or NULL for none (lora_ids is
 *                 then NULL): gate_up_A [E*S, 2 rank, hidden], gate_up_B [E*S, 2 inter, rank],
 *                 down_A [E*S, rank, inter], down_B [E*S, hidden, rank], 16-byte aligned;
 *                 slot_scale float32 [S]; slot_ranks int32 [S] or NULL (clamped to [0, rank]; the
 *                 weights past a slot's rank are never read)
 *   x             [M, ld_x], 16-byte aligned rows;  y [M, ld_y] out, aligned to its element.
 *                 y may not overlap x.
 *   topk_ids int32 [M, topk], topk_weights float32 [M, topk], lora_ids int32 [M] or NULL
 *   workspace     device scratch of mol_moe_layer_workspace_bytes(), 16-byte aligned; needs no
 *                 initial contents. Calls that may overlap must not share a workspace.
 * Requires hidden, inter, ld_x and rank to be multiples of 16 bytes' worth of elements (8
 * bf16, 4 fp32), with 4-bit weights hidden and inter multiples of group.
 * Errors: MOL_E_ARG, MOL_E_DTYPE, MOL_E_ALIGN, MOL_E_WORKSPACE, MOL_E_LIMIT (M * topk >
 * MOL_LAYER_MAX_PAIRS, topk > MOL_LAYER_MAX_TOPK, E * S + 1 > MOL_MAX_BUCKETS, rank over
 * MOL_MAX_RANK_BYTES, one expert's matrix 2 GiB or more, 2^24 work items or more in a launch). M = 0
 * is a no-op.
 * For more tokens: mol_align_block_size, mol_moe_gemm or mol_moe_gemm_q4, mol_lora_delta and
 * mol_moe_combine.
 * ------------------------------------------------------------------------------- */
#define MOL_LAYER_MAX_PAIRS 4096
#define MOL_LAYER_MAX_TOPK 64

typedef struct mol_moe_weights {
    int32_t dtype;
    int32_t group; /* 0: dense; 32, 64 or 128: 4-bit weights with group scales */
    int32_t num_experts;
    int32_t hidden;
    int32_t inter;
    int32_t reserved;
    const void *gate_up;
    const void *down;
    const void *gate_up_scales;
    const void *down_scales;
    const uint8_t *gate_up_zeros;
    const uint8_t *down_zeros;
} mol_moe_weights;

typedef struct mol_moe_adapters {
    int32_t num_slots;
    int32_t rank;
    const void *gate_up_A;
    const void *gate_up_B;
    const void *down_A;
    const void *down_B;
    const float *slot_scale;
    const int32_t *slot_ranks;
} mol_moe_adapters;

/* bytes of a layer's workspace (rank 0: no adapters), or -mol_status */
MOL_API int64_t mol_moe_layer_workspace_bytes(int32_t dtype, int32_t M, int32_t topk,
                                              int32_t hidden, int32_t inter, int32_t rank);
MOL_API mol_status mol_moe_layer(const mol_moe_weights *w, const mol_moe_adapters *adapters,
                                 const void *x, int64_t ld_x, const int32_t *topk_ids,
                                 const float *topk_weights, const int32_t *lora_ids, int32_t M,
                                 int32_t topk, void *y, int64_t ld_y, void *workspace,
                                 size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOL_H */
