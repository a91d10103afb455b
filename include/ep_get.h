/*
 * ep_get.h — C ABI of a single-GPU MoE expert-parallel token dispatch / combine.
 *
 * The EP ranks are logical partitions of one GPU's memory: rank r's tokens are
 * rows [r*T, (r+1)*T) of the inputs, and rank r's receive buffer is region r of
 * the receive tensors. Every move is a device-memory scatter or gather on the
 * caller's stream.
 *
 * Sources (DeepEP issue and pull-request pages):
 *   [P753] PR #753 "Kernel-side deterministic dispatch for the non-expand
 *          layout": Motivation, Approach, "Direct vs hybrid dispatch",
 *          Compatibility, "New API".
 *   [P690] PR #690 "Add Direct Recv X dispatch path": review comments on the
 *          copy epilogue and the buffer sizing; Summary; Implementation.
 *   [P544] PR #544 "Fix duplicate calculation of num_tokens_per_rank" (title,
 *          cited from the footer of issue #647).
 *
 * Conventions for every entry point:
 *   - Pointers named "device" must point to device memory of the current CUDA
 *     device; the caller owns and allocates every buffer, including the
 *     workspace. The library never allocates, frees or synchronises, except
 *     ep_check_error, which synchronises the given stream.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream). All work
 *     is enqueued asynchronously on it, in call order. The layout, dispatch and
 *     combine kernels are launched with programmatic stream serialization: one
 *     may be placed on the SMs while the kernel before it drains, but it waits
 *     for that kernel's completion before it reads or writes memory, so stream
 *     order holds as for any launch.
 *   - Returns EP_OK (0) or a negative EP_ERR_* code. Host-detectable errors are
 *     reported before anything is enqueued. Errors found on the device (bad
 *     top-k values; a bounded wait that ran out; in the bounds-checked build
 *     libep_get_checked.so, a row index outside its buffer) are latched in the
 *     workspace and read by ep_check_error.
 *     Unsupported combinations return EP_ERR_UNSUPPORTED; nothing is ever
 *     dropped silently.
 *   - All row pointers must be 16-byte aligned.
 */
#ifndef EP_GET_H_
#define EP_GET_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes -------------------------------------------------------- */
#define EP_OK 0
#define EP_ERR_INVALID_ARG (-1) /* bad size, null or misaligned pointer      */
#define EP_ERR_UNSUPPORTED (-2) /* valid request this library does not do    */
#define EP_ERR_WORKSPACE (-3)   /* workspace missing or smaller than needed  */
#define EP_ERR_CUDA (-4)        /* a CUDA launch or runtime call failed      */
#define EP_ERR_BAD_TOPK (-5)    /* device: top-k value < -1 or >= num_experts,
                                   or a repeated expert in the expanded layout */
#define EP_ERR_OVERFLOW (-6)    /* device: an entry did not fit its receive
                                   buffer: a packed row past recv_capacity
                                   (that entry was not written, and combine
                                   left its lane out)                        */
#define EP_ERR_TIMEOUT (-7)     /* device: a bounded wait for a bulk copy gave
                                   up (the kernel returned early; its
                                   outputs are incomplete)                   */
#define EP_ERR_BOUNDS (-8)      /* device, checked builds only
                                   (libep_get_checked.so): a computed row
                                   index fell outside its buffer; that access
                                   was skipped                               */
#define EP_ERR_NONFINITE (-9)   /* device: the router met a NaN or +inf logit or
                                   choice score (taken as -inf: not chosen)  */

/* ---- element types ------------------------------------------------------- */
#define EP_DTYPE_BF16 0
#define EP_DTYPE_FP8_E4M3 1 /* OCP E4M3 ("FN"), fp32 scale per 128 columns */
#define EP_DTYPE_FP32 2     /* router logits, and the rows in front of the norm */

/* ---- configuration --------------------------------------------------------
 * Ranks: R = num_scaleout_ranks * num_scaleup_ranks; global rank
 * r = scaleout * num_scaleup_ranks + scaleup. num_scaleout_ranks == 1 is the
 * direct layout, > 1 the hybrid row form [P753 "Direct vs hybrid dispatch"].
 * Experts: expert e lives on rank e / (num_experts / R).
 */
typedef struct ep_config {
  int32_t num_scaleout_ranks;      /* >= 1; 1 = direct                           */
  int32_t num_scaleup_ranks;       /* >= 1; R <= 64                              */
  int32_t num_experts;             /* multiple of R                              */
  int32_t num_topk;                /* K, 1..32                                   */
  int32_t num_tokens;              /* T per logical rank, 0..num_max_tokens_per_rank */
  int32_t num_max_tokens_per_rank; /* M >= 1                                     */
  int32_t hidden;                  /* H; multiple of 8 (bf16), of 128 with FP8   */
  int32_t x_dtype;                 /* EP_DTYPE_BF16, or EP_DTYPE_FP8_E4M3 (pre-cast x + x_sf) */
  int32_t recv_dtype;              /* EP_DTYPE_BF16, or EP_DTYPE_FP8_E4M3 (cast inside dispatch
                                      when x is bf16)                            */
  int32_t expand;                  /* 0 = row form, 1 = expanded per-expert blocks */
  int32_t expert_alignment;        /* >= 1: expanded blocks padded to a multiple */
  int32_t num_sms;                 /* SMs for dispatch/combine; 0 = all          */
  int32_t num_prologue_sms;        /* SMs for the layout prologue; 0 = automatic;
                                      capped at 64 [P753 "New API"]. Results never
                                      depend on it.                              */
  int32_t compact_recv;            /* row form only. 0: receive rows at their slots;
                                      1 (compact): each destination's rows packed from
                                      the start of its R*M-row window in row-block
                                      order ([P690] Direct Recv X: the entries of row
                                      block i start at the exclusive prefix
                                      recv_psum[d][i-1] of the receive counts);
                                      2 (packed): the same order with the destinations
                                      back to back in one buffer of recv_capacity rows
                                      (destination d from layout.recv_region[d]), so
                                      the receive tensors hold only what can arrive */
  int32_t zero_padding;            /* expanded only: 1 = dispatch writes zeros into the
                                      rows between each expert's lanes and the next
                                      expert_alignment boundary (and their FP8
                                      scales); 0 = those rows are left untouched  */
  int32_t sf_pack;                 /* FP8 receive only. 0: recv_sf row = G fp32 scales
                                      (amax/448). 1: packed power-of-two scales (a
                                      reading of [P690]'s num_sf_packs, whose format the
                                      pages do not give): per 128 columns one byte
                                      e+127 (UE8M0) with 2^e the smallest power of two
                                      >= amax/448 and q = e4m3(x * 2^-e); four groups
                                      per 32-bit word, group g in byte g%4 of word g/4,
                                      so a row holds ceil(G/4) words. Pre-cast FP8
                                      input then carries x_sf in the same packing.  */
  int32_t copy_path;               /* how dispatch moves rows that travel unchanged
                                      (bf16 -> bf16, pre-cast FP8): 0 = automatic
                                      (bulk copies when the input rows total
                                      at least 32 MiB, register copies below);
                                      1 = 16-byte register loads and stores; 2 = bulk
                                      copies through shared memory. Results never
                                      depend on it; the fused cast ignores it.     */
  int32_t recv_capacity;           /* packed rows only (compact_recv = 2): rows of the
                                      receive tensors; 0 = R*T*min(K, R), the most
                                      that can arrive (every token has at most min(K,R)
                                      destinations). An entry past it is not written
                                      and latches EP_ERR_OVERFLOW; layout.recv_region[R]
                                      gives the exact count after the layout.      */
} ep_config_t;

/* ---- dispatch layout (all device pointers, int32 unless noted) -------------
 * Row form: destination d's region of the receive tensors has R*M rows; source
 * s owns the M rows starting at row_block(s)*M, where row_block(s) = s
 * (direct) or scaleup(s)*num_scaleout_ranks + scaleout(s) (hybrid: segment =
 * source scale-up rank, in-segment offset = source scale-out rank * M + slot)
 * [P753 Approach; "Direct vs hybrid dispatch"].
 */
typedef struct ep_layout {
  int32_t* num_tokens_per_rank;   /* [R src][R dst]: tokens of src reaching dst,
                                     once per token [P544]                      */
  int32_t* num_tokens_per_expert; /* [R src][E]: valid lanes per expert         */
  uint8_t* is_token_in_rank;      /* [R][T][R dst]: 0/1                          */
  int32_t* slot_map;              /* [R][T][K]: row inside the destination region =
                                     row_block(src)*M + the source's running count of
                                     deduplicated entries to that destination in token
                                     order; lanes to the same destination share it;
                                     -1 for masked lanes [P753 Approach]         */
  int32_t* recv_cnt;              /* [R dst][R src] = num_tokens_per_rank transposed */
  int32_t* recv_psum;             /* [R dst][R row blocks]: inclusive prefix sums of
                                     recv_cnt in row-block order [P753 "Direct vs
                                     hybrid dispatch": per-source receive counts] */
  /* expanded layout only (may be NULL when expand == 0): per destination, per
     local expert j, a block of rows holding that expert's lanes in (source rank,
     token) order, padded to expert_alignment; regions concatenated by rank. */
  int32_t* exp_cnt;    /* [R][L]: lanes per (destination, local expert)         */
  int32_t* exp_base;   /* [R][L+1]: block starts inside the region; [L] = size  */
  int32_t* exp_region; /* [R+1]: first row of each region; [R] = total rows     */
  int32_t* exp_pos;    /* [R][T][K]: row of the lane inside its destination's
                          region, -1 for masked lanes                          */
  int32_t* recv_region; /* [R+1] (may be NULL unless compact_recv = 2): first
                           packed row of each destination = the entries all
                           destinations before it receive; [R] = total entries */
} ep_layout_t;

/* ---- receive buffers (device pointers) -------------------------------------
 * Row form: recv_x/recv_sf and the sidecars' rows are indexed d*R*M + slot;
 * compact (compact_recv = 1): d*R*M + recv_psum[d][rb-1] + slot - rb*M with
 * rb = slot / M (recv_psum[d][-1] = 0), so destination d's rows are
 * [d*R*M, d*R*M + sum_s recv_cnt[d][s]); packed (compact_recv = 2):
 * recv_region[d] + recv_psum[d][rb-1] + slot - rb*M, so destination d's rows
 * are [recv_region[d], recv_region[d+1]) and all tensors have ep_recv_rows()
 * rows. Expanded: recv_x and recv_sf rows are indexed exp_region[d] + exp_pos;
 * the sidecars stay in the row form. Rows no entry fills are left untouched.
 * recv_topk_idx, recv_topk_weights and recv_src_metadata may be NULL (not
 * written).
 */
typedef struct ep_recv {
  void* recv_x;                /* [recv_x_rows][H] bf16 or e4m3                 */
  float* recv_sf;              /* [recv_x_rows][H/128] fp32, or [recv_x_rows][ceil(H/512)]
                                  packed words with sf_pack (FP8 receive only)   */
  int64_t* recv_topk_idx;      /* [R][R*M][K] (packed: [ep_recv_rows][K]):
                                  destination-local expert or -1                 */
  float* recv_topk_weights;    /* same rows x K: weight, or 0 off this destination */
  int32_t* recv_src_metadata;  /* same rows x (2+K): {src rank, src token,
                                  dst_tensor_idx[K]}; field 2+k = expanded row of
                                  lane k in this destination's region, else -1
                                  [P690 copy-epilogue review]                   */
  int64_t recv_x_rows;         /* capacity of recv_x in rows, >= ep_recv_rows()  */
} ep_recv_t;

/* Workspace bytes the three entry points need for this configuration (the
 * library's own convention: the pages' buffers are transport windows with no
 * single-GPU counterpart): a 256-byte header (the device error word, the
 * layout's arrival counter, and the work queues from which the dispatch and
 * combine warps take their tokens), plus per-(source, expert) offsets when
 * expanding. The workspace must be zero-filled before its first use
 * (ep_workspace_init or a zeroing allocator); afterwards every kernel returns
 * its counters to zero itself. One workspace serves one stream at a time. */
size_t ep_workspace_bytes(const ep_config_t* cfg);

/* Rows the receive buffer recv_x needs: R*R*M (row form and compact; the
 * per-destination window of [P690]'s buffer sizing times R), recv_capacity or
 * R*T*min(K, R) (packed), or R*T*K + E*(expert_alignment-1) (expanded upper
 * bound). Returns -1 for an invalid configuration. */
int64_t ep_recv_rows(const ep_config_t* cfg);

/* Zero the workspace on `stream` (the library's own convention). */
int ep_workspace_init(void* workspace, size_t workspace_bytes, void* stream);

/* Dispatch layout [P753 Motivation, Approach]: turns topk_idx (device, int64
 * [R][T][K]; -1 = masked lane) into the counts, the per-lane slots and, when
 * expanding, the per-expert positions of `layout` (all device outputs). One
 * kernel with a thread-block cluster per source rank: per-warp counts, a scan
 * of the CTAs' counts through distributed shared memory, then per-lane slots;
 * its last CTA writes the receive prefix sums (and recv_region). The expanded
 * layout adds two small kernels (the per-expert scan across sources, then the
 * final positions). The result is a pure function of topk_idx. */
int ep_get_dispatch_layout(const ep_config_t* cfg, const int64_t* topk_idx,
                           const ep_layout_t* layout, void* workspace,
                           size_t workspace_bytes, void* stream);

/* Size of the fixed scratch array used by ep_get_dispatch_layout_noalloc. */
#define EP_NOALLOC_SCRATCH_BYTES (1u << 20)

/* ep_get_dispatch_layout for callers that cannot allocate device memory (for
 * example plugins of inference engines that are handed only their input and
 * output buffers, or latency-critical code where cudaMalloc is not allowed).
 * No counterpart on the DeepEP pages: it is the same layout with the workspace
 * replaced by a fixed array of EP_NOALLOC_SCRATCH_BYTES inside the library,
 * which every GPU that loads the library keeps until the process exits.
 *   - Outputs, layout and errors for invalid arguments are those of
 *     ep_get_dispatch_layout; a configuration whose ep_workspace_bytes exceeds
 *     EP_NOALLOC_SCRATCH_BYTES returns EP_ERR_WORKSPACE.
 *   - Allocates nothing. The first call in a CUDA context (that context
 *     current) looks up the array's device address; make it before any stream
 *     capture. A device reset gives a new context, and the next call looks the
 *     address up again.
 *   - All calls share the array: each call, once its arguments have passed
 *     the checks, clears the array's error bits and counter on `stream`
 *     first; calls that overlap on the GPU race on it.
 *   - Invalid top-k values are treated as masked lanes, as in
 *     ep_get_dispatch_layout, and latched in the array's error word, which
 *     ep_check_error_noalloc reads. */
int ep_get_dispatch_layout_noalloc(const ep_config_t* cfg, const int64_t* topk_idx,
                                   const ep_layout_t* layout, void* stream);

/* ep_check_error for ep_get_dispatch_layout_noalloc (no counterpart on the
 * pages): synchronises `stream`, returns the first device-detected error the
 * allocation-free layout latched in the library's array since the last call
 * (EP_OK if none) and clears it. Allocates nothing; shares the array, and its
 * race with overlapping calls, with ep_get_dispatch_layout_noalloc. */
int ep_check_error_noalloc(void* stream);

/* Dispatch: for every deduplicated (token, destination) entry writes the
 * token's hidden row into the destination's receive rows at its slot (row
 * form) or, expanded, one row per valid lane at its position; plus the
 * sidecars [P753 Approach; P690 Summary/Implementation].
 *   x: device [R][T][H] bf16 (x_dtype BF16) or e4m3 codes (FP8).
 *   x_sf: device [R][T][H/128] fp32, FP8 input only (else NULL).
 *   recv_dtype FP8 with bf16 x casts inside the copy: per 128 columns,
 *   amax = max(max|x|, 1e-4), sf = amax/448, q = e4m3_rn_satfinite(x*(448/amax)).
 *   topk_idx / topk_weights: device [R][T][K] int64 / fp32.
 * `layout` must come from ep_get_dispatch_layout with the same cfg/topk_idx. */
int ep_dispatch(const ep_config_t* cfg, const ep_layout_t* layout, const void* x,
                const float* x_sf, const int64_t* topk_idx, const float* topk_weights,
                const ep_recv_t* recv, void* workspace, size_t workspace_bytes,
                void* stream);

/* Combine: out[s][t] = bf16_rn(acc), acc = +0 then, for k in lane order over
 * the valid lanes, acc = fma(topk_weights[s][t][k], y[row of lane k], acc),
 * in fp32. y: device bf16 expert outputs in the receive layout (row form or
 * compact [R][R*M][H], or expanded [rows][H]), at least ep_recv_rows(cfg)
 * rows; out: device bf16 [R][T][H]. The result is bitwise reproducible. */
int ep_combine(const ep_config_t* cfg, const ep_layout_t* layout, const uint16_t* y,
               const int64_t* topk_idx, const float* topk_weights, uint16_t* out,
               void* workspace, size_t workspace_bytes, void* stream);

/* ---- comparison path: the design PR #753 replaces ----------------------------
 * [P753 Motivation] Before kernel-side slots, a sender took its destination slot
 * with an atomicAdd on a shared counter, so the order of a source's rows inside
 * a destination depended on the race between warps, and EPHandle.deterministic_sort
 * restored a reproducible order afterwards by sorting the received tokens by
 * source token and permuting every order-dependent tensor. These two entry points
 * reproduce that path (row form only, not compact) so it can be measured against
 * ep_get_dispatch_layout + ep_dispatch; after the sort the buffers equal the
 * deterministic dispatch's bit for bit.
 *
 * ep_dispatch_atomic: ep_dispatch without a layout. send_counters: device int32
 * [R src][R dst], zeroed on `stream` by the call, then left holding how many
 * rows each source sent each destination. Rows land in the source's row block
 * of the destination region in race order. The workspace (as for ep_dispatch)
 * carries the work queue that spreads the tokens over the warps. */
int ep_dispatch_atomic(const ep_config_t* cfg, const void* x, const float* x_sf,
                       const int64_t* topk_idx, const float* topk_weights, const ep_recv_t* recv,
                       int32_t* send_counters, void* workspace, size_t workspace_bytes, void* stream);

/* ep_deterministic_sort: sorts every (destination, row block) segment of `recv`
 * (filled by ep_dispatch_atomic; the sidecars must be present: the key is the
 * metadata's source token) and writes rows and sidecars in that order to
 * `sorted` (same shapes). num_max_tokens_per_rank <= 8192. */
int ep_deterministic_sort(const ep_config_t* cfg, const ep_recv_t* recv,
                          const int32_t* send_counters, const ep_recv_t* sorted, void* stream);

/* ---- router -------------------------------------------------------------------
 * What stands before the dispatch (no counterpart on the DeepEP pages, which take
 * topk_idx and topk_weights as given): the chosen experts of every token with
 * their weights, in the form the dispatch and combine read, the lanes per expert
 * and the balance loss; and the gradient of the logits.
 *
 * Tokens come in num_segments segments of num_tokens each (the source ranks, or
 * sequences); the loss is taken over each segment. N = num_segments * num_tokens.
 */
#define EP_SCORE_SOFTMAX 0
#define EP_SCORE_SIGMOID 1

typedef struct ep_route_config {
  int32_t num_segments; /* B >= 1                                                  */
  int32_t num_tokens;   /* T >= 0 per segment; B * T * num_topk below 2^31         */
  int32_t num_experts;  /* E, 1..4096                                              */
  int32_t num_topk;     /* K, 1..32, at most E                                     */
  int32_t logits_dtype; /* EP_DTYPE_FP32 or EP_DTYPE_BF16 (logits and d_logits)    */
  int32_t score;        /* s = softmax(l) or sigmoid(l) of a token's logits l      */
  int32_t num_groups;   /* G: 0 or 1 = none; else E in G groups of neighbours, 2 experts
                           at least each, G <= 32                                  */
  int32_t topk_groups;  /* groups a token may choose from, 1..G, holding K experts at
                           least (ignored without groups)                          */
  int32_t normalize;    /* 1: weights divided by the sum of s over the chosen (taken
                           of logarithms where sigmoids are tiny; 0 where the chosen s
                           are all 0 in 64 bits: logits below -745)                */
  float scale;          /* every weight times this (finite)                        */
} ep_route_config_t;

/* Device outputs. The last four are the statistics: all present, or all NULL (a
 * serving step needs none). */
typedef struct ep_route {
  int64_t* topk_idx;     /* [N][K]: chosen experts, best first; -1 where none is left */
  float* topk_weights;   /* [N][K]: scale * s (/ sum); 0 where topk_idx is -1       */
  int32_t* expert_count; /* [B][E]: lanes to each expert                            */
  float* prob_sum;       /* [B][E]: sum over the segment's tokens of p = s (softmax)
                            or s / sum s (sigmoid)                                  */
  int32_t* num_valid;    /* [B]: tokens the mask leaves                             */
  float* balance_loss;   /* [1]: mean over the segments of sum_e (E count_e / (K n))
                            (prob_sum_e / n), n = num_valid; 0 for an empty segment */
} ep_route_t;

/* Workspace bytes of ep_route and ep_route_grad (0 for an invalid configuration).
 * Zero-filled once before first use (ep_workspace_init), as the others (it may then
 * serve any configuration that fits it); one stream at a time; errors are read by
 * ep_check_error. */
size_t ep_route_workspace_bytes(const ep_route_config_t* cfg);

/* Router. logits: device [N][E], 16-byte aligned. choice_bias: device fp32 [E] or
 * NULL: added to the score the choice is made by (l for softmax, s for sigmoid),
 * not to the weights. token_mask: device uint8 [N] or NULL; 0 = padding: idx -1,
 * weights 0, not counted, its logits are not read for anything.
 *   - The K experts of largest choice score in order, ties to the lowest expert;
 *     with groups, among the topk_groups groups whose two best choice scores have the
 *     largest fp32 sum, ties to the lowest group.
 *   - With softmax scores the choice score is the logit. Without groups and bias that chooses
 *     the largest probabilities. A bias is added to logits, and groups are ranked by sums
 *     of logits: a router trained with a bias on probabilities, or with groups ranked by
 *     sums of probabilities, chooses differently and is not what this computes.
 *   - An expert whose logit or choice score is -inf is never chosen; lanes for which
 *     no expert is left are -1. NaN and +inf are taken as -inf and latch
 *     EP_ERR_NONFINITE.
 *   - Results are bitwise reproducible. Without tokens the statistics are zeros. */
int ep_route(const ep_route_config_t* cfg, const void* logits, const float* choice_bias,
             const uint8_t* token_mask, const ep_route_t* out, void* workspace,
             size_t workspace_bytes, void* stream);

/* Gradient of the logits through the weights and the loss; the choice and the
 * counts are constants. `route` holds ep_route's outputs (topk_idx; with d_loss
 * also expert_count and num_valid). d_weights: device fp32 [N][K] or NULL (zero); what
 * stands where topk_idx is -1 is not used.
 * d_loss: device fp32 [1], the gradient of balance_loss (its coefficient included),
 * or NULL (zero). d_logits: device [N][E] of the logits' type, every element
 * written (zero for padding tokens), 16-byte aligned. A topk_idx outside [-1, E)
 * latches EP_ERR_BAD_TOPK and is treated as masked. */
int ep_route_grad(const ep_route_config_t* cfg, const void* logits, const uint8_t* token_mask,
                  const ep_route_t* route, const float* d_weights, const float* d_loss,
                  void* d_logits, void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of ep_combine: for d_out (device bf16 [R][T][H]),
 *   d_weights[s][t][k] = <d_out[s][t], y[row of lane k]> (fp32; 0 for a masked lane),
 *   d_y[row] = bf16_rn((sum of topk_weights over the token's lanes on that row) *
 *              d_out[s][t]); rows that no lane reads are left untouched.
 * Either of d_y, d_weights may be NULL; y may be NULL when d_weights is. The layout,
 * y, topk_idx, topk_weights, workspace and errors are ep_combine's, for every
 * receive layout. Bitwise reproducible. (Where every lane has a row of its own, the
 * expanded layout, the gradient of the dispatch itself is ep_combine with weights 1.) */
int ep_combine_grad(const ep_config_t* cfg, const ep_layout_t* layout, const uint16_t* y,
                    const int64_t* topk_idx, const float* topk_weights, const uint16_t* d_out,
                    uint16_t* d_y, float* d_weights, void* workspace, size_t workspace_bytes,
                    void* stream);

/* ---- the experts' products --------------------------------------------------------
 * What stands between dispatch and combine: the rows of every expert's block of an
 * expanded layout times that expert's matrix, with bias, activation and residual:
 *   z[r] = x[r] W_g^T + b_g,   out[r] = act(z[r]) + residual[r]     for r in block g
 * (gated: z has 2 N columns, out = silu(z[:, :N]) * z[:, N:] + residual). Products are
 * of bf16 values, summed in fp32; the activation is taken of the fp32 sum; z and out
 * are rounded once. Rows outside the blocks' lanes are neither read for a result nor
 * written. layout = NULL: one group of all `rows` rows (a dense product, such as a
 * shared expert), with num_ranks = num_experts = 1. Every wait in the kernels is
 * bounded; one that gives up latches EP_ERR_TIMEOUT and leaves outputs incomplete.
 */
#define EP_ACT_NONE 0
#define EP_ACT_RELU 1   /* max(z, 0); NaN stays NaN, as under the others */
#define EP_ACT_SILU 2   /* z / (1 + exp(-z))            */
#define EP_ACT_GELU 3   /* z * (1 + erf(z / sqrt 2)) / 2 */
#define EP_ACT_SWIGLU 4 /* gated: silu(z1) * z2          */

typedef struct ep_product_config {
  int32_t num_ranks;    /* R of the layout                                         */
  int32_t num_experts;  /* E, a multiple of R, 1..4096                             */
  int64_t rows;         /* rows of x, z, out, residual, 0..2^31-1 (ep_recv_rows of the
                           dispatch); a block past them is cut and latches EP_ERR_OVERFLOW,
                           as do blocks that overlap (some of their rows are left out)  */
  int32_t in_features;  /* K, a multiple of 8 (of 128 with FP8), up to 2^20         */
  int32_t out_features; /* N of out, a multiple of 8, up to 2^20                    */
  int32_t activation;   /* EP_ACT_*                                                 */
  int32_t x_dtype;      /* EP_DTYPE_BF16, or EP_DTYPE_FP8_E4M3: the rows and x_sf of an
                           FP8 dispatch (each element is code * scale, not rounded;
                           forward only)                                            */
  int32_t sf_pack;      /* x_sf as ep_config_t.sf_pack                              */
  int32_t num_sms;      /* SMs to use; 0 = all. Results do not depend on it. (d_weight
                           is computed by pairs of SMs: it takes two for 1)         */
} ep_product_config_t;

/* Workspace bytes of ep_expert_product (grad = 0) or ep_expert_product_grad (1); 0 for
 * an invalid configuration. Its 256-byte header is zero-filled once before first use
 * (every call leaves its counters zero); one stream at a time; errors are read by
 * ep_check_error. */
size_t ep_product_workspace_bytes(const ep_product_config_t* cfg, int32_t grad);

/* Forward. All device pointers, rows dense and 16-byte aligned: x [rows][K], weight
 * bf16 [E][Z][K] (Z = N, or 2 N gated: the N gate rows, then the N others), bias bf16
 * [E][Z] or NULL, residual bf16 [rows][N] or NULL (it may be out itself), z bf16
 * [rows][Z] or NULL (kept for the gradient), out bf16 [rows][N]. x_sf: the FP8 rows'
 * scales, else NULL. Bitwise reproducible. */
int ep_expert_product(const ep_product_config_t* cfg, const ep_layout_t* layout, const void* x,
                      const float* x_sf, const uint16_t* weight, const uint16_t* bias,
                      const uint16_t* residual, uint16_t* z, uint16_t* out, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Gradients for d_out (bf16 [rows][N]), with dz = d_out * act'(z) from the kept z
 * (NULL allowed when the activation is none):
 *   d_x[r] = dz[r] W_g (bf16), d_weight_g = sum over the block's rows of dz[r]^T x[r]
 *   (bf16 [E][Z][K], zeros for an empty block), d_bias_g = sum of dz (fp32 [E][Z]).
 * Any of the three may be NULL; x is needed for d_weight, weight for d_x. dz enters the
 * products rounded to bf16 and d_bias unrounded. The gradient of the residual is
 * d_out itself. bf16 x only. Bitwise reproducible. */
int ep_expert_product_grad(const ep_product_config_t* cfg, const ep_layout_t* layout,
                           const uint16_t* x, const uint16_t* weight, const uint16_t* z,
                           const uint16_t* d_out, uint16_t* d_x, uint16_t* d_weight,
                           float* d_bias, void* workspace, size_t workspace_bytes, void* stream);

/* ---- norm in front of the router ----------------------------------------------------
 * (No counterpart on the DeepEP pages.) The residual's addition and the root-mean-square
 * norm, in bf16 for the router and the experts, and as the FP8 rows with scales that
 * ep_dispatch takes (x_dtype EP_DTYPE_FP8_E4M3):
 *   s = x + residual,   y = s / sqrt(mean of s^2 over the row + eps) * weight
 */
typedef struct ep_norm_config {
  int64_t rows;    /* 0..2^31-1                                                       */
  int32_t hidden;  /* H, a multiple of 8 (of 128 with codes), up to 16384             */
  int32_t x_dtype; /* of x, residual, sum, d_sum and d_x: EP_DTYPE_BF16 or EP_DTYPE_FP32 */
  int32_t sf_pack; /* the scales' format, as ep_config_t.sf_pack                      */
  float eps;       /* 1e-20 to 1e38                                                   */
} ep_norm_config_t;

/* Forward. Device pointers, rows dense and 16-byte aligned: x [rows][H]; residual the same or
 * NULL; weight bf16 [H] or NULL (ones); sum [rows][H] or NULL: s, rounded to x's type (it
 * may be x or residual itself); y bf16 [rows][H] or NULL; codes uint8 [rows][H] and sf
 * (fp32 [rows][H/128], or [rows][ceil(H/512)] packed words) or both NULL; y or codes is
 * there. The norm is taken of s in fp32, before it is rounded; codes are made of y before it is
 * rounded, as the dispatch's cast makes them of bf16. Sums of squares past fp32's range
 * are taken of smaller values. A NaN makes its row NaN, an infinity too (zeros beside it). */
int ep_norm(const ep_norm_config_t* cfg, const void* x, const void* residual, const uint16_t* weight, void* sum,
            uint16_t* y, uint8_t* codes, float* sf, void* stream);

/* Workspace bytes of ep_norm_grad (0 for an invalid configuration). Its 256-byte header is zero-filled
 * once before first use; one stream at a time; errors (a bounded wait that gave up) are read by
 * ep_check_error. */
size_t ep_norm_workspace_bytes(const ep_norm_config_t* cfg);

/* Gradients for d_y (bf16 [rows][H]), from the kept sum: with q = 1 / sqrt(mean s^2 + eps),
 * n = s q and t = d_y weight,
 *   d_x = q (t - n mean(t n)) + d_sum   (also the residual's gradient),
 *   d_weight = sum over the rows of d_y n (fp32 [H]).
 * d_sum: what arrives at the sum itself, [rows][H] of x's type, or NULL (zero); d_x may take its
 * place. d_x or d_weight may be NULL. token_mask: uint8 [rows] or NULL; 0 = padding: d_x is
 * zero there, its other tensors are not read. Codes pass gradients on as if they were not
 * rounded. Bitwise reproducible. */
int ep_norm_grad(const ep_norm_config_t* cfg, const void* sum, const uint16_t* weight, const uint8_t* token_mask,
                 const uint16_t* d_y, const void* d_sum, void* d_x, float* d_weight, void* workspace,
                 size_t workspace_bytes, void* stream);

/* ---- rows kept in 8 bits for the backward pass ----------------------------------------
 * (No counterpart on the DeepEP pages.) The rows of an expanded layout's blocks in the form of the
 * dispatch's FP8 rows, half of bf16's bytes: z of the experts' products, or the rows that were
 * dispatched as FP8 (those are in this form already). Rows outside the blocks' lanes are
 * neither read for a result nor written. layout = NULL: one group of all rows, with
 * num_ranks = num_experts = 1; blocks that leave the rows or overlap are cut as in the products
 * and latch EP_ERR_OVERFLOW. Each kept value is off by at most 2^-4 of itself, or of the
 * least step of its 128 columns (2^-10 of their scale).
 */
typedef struct ep_checkpoint_config {
  int32_t num_ranks;   /* R of the layout                                              */
  int32_t num_experts; /* E, a multiple of R, 1..4096                                  */
  int64_t rows;        /* 0..2^31-257                                                  */
  int32_t features;    /* F, columns of the kept rows (Z of the product), a multiple of
                          128, up to 2^21                                              */
  int32_t activation;  /* EP_ACT_*, ep_checkpoint_grad only (gated: F = 2 N)           */
  int32_t sf_pack;     /* the scales' format, as ep_config_t.sf_pack                   */
} ep_checkpoint_config_t;

/* Workspace bytes of the three calls (0 for an invalid configuration). Its 256-byte header is
 * zero-filled once before first use (every call leaves its counters zero); one stream at a
 * time; errors are read by ep_check_error. */
size_t ep_checkpoint_workspace_bytes(const ep_checkpoint_config_t* cfg);

/* x bf16 [rows][F] -> codes uint8 [rows][F], sf fp32 [rows][F/128] or packed words
 * [rows][ceil(F/512)]: the codes and scales of ep_dispatch's cast, bit for bit. */
int ep_checkpoint(const ep_checkpoint_config_t* cfg, const ep_layout_t* layout, const uint16_t* x, uint8_t* codes, float* sf,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Back: x = bf16_rn(code * scale), exact with packed scales (down to bf16's least numbers), such as
 * the x that ep_expert_product_grad needs for d_weight. */
int ep_checkpoint_rows(const ep_checkpoint_config_t* cfg, const ep_layout_t* layout, const uint8_t* codes, const float* sf,
                       uint16_t* x, void* workspace, size_t workspace_bytes, void* stream);

/* The backward pass through the activation, from kept z = code * scale (fp32, not rounded) and
 * d_h (bf16 [rows][N]): h = act(z) (bf16 [rows][N]: x of the next product's d_weight, so that it
 * need not be kept), d_z = d_h act'(z) (bf16 [rows][F]: d_out of the product's own gradient
 * with EP_ACT_NONE), d_bias_g = column sums of the unrounded d_z over the block (fp32
 * [E][F], zeros for an empty block). Any of the three may be NULL. Bitwise reproducible. */
int ep_checkpoint_grad(const ep_checkpoint_config_t* cfg, const ep_layout_t* layout, const uint8_t* codes, const float* sf,
                       const uint16_t* d_h, uint16_t* h, uint16_t* d_z, float* d_bias, void* workspace,
                       size_t workspace_bytes, void* stream);

/* ---- the experts' layer of a few tokens ------------------------------------------------
 * (No counterpart on the DeepEP pages.) What dispatch, both products of each expert and combine
 * compute for a serving step of up to 64 tokens on one rank, straight from the router's choice, in
 * two kernels that read each chosen expert's matrices once for every 16 of its tokens:
 *   h = act(x_t W_up[e]^T + b_up[e]),   out_t = sum over the lanes k of topk_weights[t][k] *
 *   (h W_down[e]^T + b_down[e]) + residual_t          with e = topk_idx[t][k]
 * Sums are fp32; h is rounded to bf16 as between the products (for up to 4 tokens to the sum of
 * two bf16, off by 2^-16 of itself at most), out once; the lanes' results are not rounded.
 * ep_dispatch and ep_expert_product take any number of tokens, and are faster from about 8 tokens
 * an expert on.
 */
typedef struct ep_layer_config {
  int32_t num_tokens;   /* T, 0..64                                                      */
  int32_t num_experts;  /* E, 1..4096                                                    */
  int32_t num_topk;     /* K, 1..32                                                      */
  int32_t hidden;       /* H, a multiple of 8 (of 128 with FP8 matrices), up to 2^20     */
  int32_t inner;        /* I, a multiple of 8 (of 128 with FP8 matrices), up to 2^20     */
  int32_t activation;   /* EP_ACT_*; gated: up has Z = 2 I rows, the I gate rows first   */
  int32_t weight_dtype; /* EP_DTYPE_BF16, or EP_DTYPE_FP8_E4M3: codes with an fp32 scale
                           for every 128 x 128 of a matrix                               */
  int32_t num_sms;      /* SMs to use; 0 = all. Results do not depend on it.             */
} ep_layer_config_t;

/* Workspace bytes (0 for an invalid configuration). Its 256-byte header is zero-filled once before first
 * use, and it may then serve any configuration that fits it; one stream at a time; errors are read by
 * ep_check_error. */
size_t ep_layer_workspace_bytes(const ep_layer_config_t* cfg);

/* Device pointers, rows dense and 16-byte aligned: x bf16 [T][H], topk_idx int64 [T][K] and
 * topk_weights fp32 [T][K] as ep_route writes them (-1: no expert; other values outside [0, E)
 * latch EP_ERR_BAD_TOPK and count as -1; a weight where there is no expert is not used; an
 * expert twice counts with both weights), up [E][Z][H] and down [E][H][I] bf16, or codes with
 * up_sf fp32 [E][ceil(Z/128)][H/128] and down_sf [E][H/128][I/128] (else NULL), up_bias bf16
 * [E][Z], down_bias bf16 [E][H], residual bf16 [T][H] or NULL each (residual may be out itself,
 * and out may be x), out bf16 [T][H]. Matrices of experts that no token chose are not read.
 * A token without an expert gets its residual, or 0. Bitwise reproducible. */
int ep_expert_layer(const ep_layer_config_t* cfg, const uint16_t* x, const int64_t* topk_idx, const float* topk_weights,
                    const void* up, const float* up_sf, const uint16_t* up_bias, const void* down, const float* down_sf,
                    const uint16_t* down_bias, const uint16_t* residual, uint16_t* out, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Synchronises `stream`, returns the first device-detected error latched in
 * the workspace since the last call (EP_OK if none) and clears it. The
 * library's own convention (the pages print and continue on a device error;
 * PR #690's review asks that nothing be dropped silently). */
int ep_check_error(void* workspace, void* stream);

/* Human-readable name of a status code (static storage; the library's own). */
const char* ep_status_string(int status);

/* Diagnostics: the device's fp32 -> e4m3 (round to nearest even, saturating)
 * and fp32 -> bf16 (round to nearest even) conversions used by the kernels,
 * applied to the binary32 bit patterns first .. first+n-1; out is device
 * memory of n bytes / n uint16. */
int ep_diag_e4m3_of_bits(uint32_t first, int64_t n, uint8_t* out, void* stream);
int ep_diag_bf16_of_bits(uint32_t first, int64_t n, uint16_t* out, void* stream);

/* Diagnostic copy for the bandwidth ceiling of a one-read, many-write stream
 * (no counterpart on the pages; the benchmark times it beside the dispatch,
 * whose scatter reads each token row once and writes it to each destination).
 * Row r of `src` (rows x row_bytes, 16-byte aligned) is read once and
 * written to rows floor(r*fan_num/fan_den) .. floor((r+1)*fan_num/fan_den) - 1
 * of `dst` (16-byte aligned, floor(rows*fan_num/fan_den) rows of row_bytes;
 * the caller owns both). Either may be device memory or pinned host memory the
 * device addresses directly (the benchmark times the host link that way). row_bytes: a positive multiple of 16;
 * 0 <= fan_num <= 2^20, fan_den >= 1, 0 <= rows <= 2^40; num_sms: SMs the grid
 * is sized for (0 = all). method 0: 16-byte register loads and stores; method
 * 1: bulk copies through shared memory (row_bytes <= 16384, else
 * EP_ERR_UNSUPPORTED). Returns EP_ERR_INVALID_ARG for any other argument,
 * EP_ERR_CUDA if the launch fails; asynchronous on `stream`. */
int ep_diag_copy_fanout(const void* src, void* dst, int64_t rows, int32_t row_bytes, int32_t fan_num,
                        int32_t fan_den, int32_t num_sms, int32_t method, void* stream);

/* Diagnostic for the bounded waits (no counterpart on the pages): one warp
 * starts a bulk load of `bytes` (0..4096, a multiple of 16) from `src` (device,
 * 16-byte aligned; may be null when bytes is 0), waits at most `rounds`
 * (<= 2^20) try_wait rounds on an mbarrier that nothing completes, drains the
 * load and latches the timeout bit in `workspace` (256-byte aligned), exactly
 * as the bulk-copy dispatch does when a wait runs out; ep_check_error then
 * returns EP_ERR_TIMEOUT. Asynchronous on `stream`. */
int ep_diag_wait_timeout(void* workspace, const void* src, int32_t bytes, uint32_t rounds, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_GET_H_ */
