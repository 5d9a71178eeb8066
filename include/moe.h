/*
 * moe.h - C ABI of libmoe: the hot path of one expert-parallel MoE layer on one GB300 GPU.
 *
 * The layer (router -> dispatch -> grouped SwiGLU expert GEMMs + shared expert -> combine) is
 * the one described in "7.13 Serving Mixture-of-Experts: Expert Parallelism & All-to-All
 * Inference" (llm-stack-book), section "Expert Parallelism Mechanics: Dispatch, Compute,
 * Combine", with the DeepSeek-V3 router of "Mixture-of-experts serving" (learn-kernels),
 * paragraphs 1 and 3, and the receive-buffer design of "One-Sided Expert-Parallel All-to-All
 * for Mixture-of-Experts Inference over NVLink" (abstract): every source pushes its rows into
 * rank-major buffers with no metadata exchange first, and the grouped GEMMs read those buffers
 * in place. The expert-parallel ranks are logical: R partitions of this GPU's memory.
 *
 * Conventions for every entry point
 *  - All array pointers are DEVICE pointers, allocated and owned by the caller. The library
 *    allocates nothing and keeps no state between calls except cached kernel attributes and
 *    the driver entry point it uses to encode TMA tensor maps.
 *  - Work is enqueued on `stream` and the call returns at once (asynchronous). No call
 *    synchronises with the host or copies device memory to the host, except
 *    moe_read_status, which says so.
 *  - Arrays are dense and row-major with the shapes given. bf16 is IEEE bfloat16, e4m3 is the
 *    8-bit float with 4 exponent bits (bias 7) and 3 mantissa bits (largest finite 448).
 *    Device pointers must be 16-byte aligned.
 *  - Return value: MOE_OK, or an MOE_ERR_* code describing the first failed check; nothing
 *    is enqueued when a check fails. moe_strerror() names the code.
 *  - Errors found on the device (a wait that ran out, a bounds check) are OR-ed into a status
 *    word at the start of the workspace `ws`; read it with moe_read_status().
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 3

/* Return codes */
#define MOE_OK 0
#define MOE_ERR_INVALID_ARG 1  /* a shape constraint failed or a required pointer is NULL */
#define MOE_ERR_UNSUPPORTED 2  /* valid MoE shape outside what these kernels implement */
#define MOE_ERR_MISALIGNED 3   /* a device pointer is not 16-byte aligned */
#define MOE_ERR_CUDA 4         /* a CUDA runtime/driver call or a kernel launch failed */

/* Device status bits (moe_read_status) */
#define MOE_DEV_TIMEOUT 1u     /* a bounded wait inside a kernel gave up; outputs invalid */
#define MOE_DEV_BOUNDS 2u      /* an index read from device memory was out of range */
#define MOE_DEV_SCALE 4u       /* MOE_FP8_E4M3_POW2: a weight block scale is not a power of two
                                  (not positive, not finite, or with mantissa bits); the GEMM
                                  applied 2^(its exponent field - 127) in its place */

#define MOE_DEV_NONFINITE 8u   /* moe_adamw: the gradients' norm is not finite; step left out */

/* Element formats */
#define MOE_BF16 0
#define MOE_FP8_E4M3 1       /* e4m3 with fp32 block scales: 1x128 for activations (scale =
                                amax / 448), 128x128 for weights (any positive scales) */
#define MOE_FP8_E4M3_POW2 2  /* e4m3 with power-of-two fp32 block scales: the same blocks, each
                                activation scale the smallest power of two 2^e with
                                amax <= 448 * 2^e (e in [-126, 127], 1 for an all-zero block);
                                the weight scales must be powers of two too. The grouped GEMMs
                                apply the scales in the tensor core (block-scaled MMA) instead
                                of promoting each 128-K block's partial sums. These kernels
                                take d % 256 == 0, d <= 8192 and d_ff <= 8192 in this format
                                (MOE_ERR_UNSUPPORTED otherwise). */

/* Number of events moe_layer records when given an event array (see moe_layer). */
#define MOE_LAYER_EVENTS 7

/* Shape of one MoE layer. Notation of the pages: T tokens of width d, E routed experts, top-k
 * routing with n_group groups of which topk_group are kept, SwiGLU experts of width d_ff,
 * one shared expert of width d_ff_shared, R logical expert-parallel ranks. */
typedef struct moe_cfg {
  int32_t T;            /* tokens in the batch, all logical ranks together; T % R == 0 */
  int32_t d;            /* model width; d % 128 == 0 */
  int32_t E;            /* routed experts; E % R == 0, E % n_group == 0, E <= 1024 */
  int32_t k;            /* experts per token; 1 <= k <= min(32, topk_group * E / n_group) */
  int32_t n_group;      /* expert groups (contiguous blocks of E/n_group experts), <= 64 */
  int32_t topk_group;   /* groups kept per token; 1 <= topk_group <= n_group */
  int32_t d_ff;         /* routed expert SwiGLU width; d_ff % 128 == 0 */
  int32_t d_ff_shared;  /* shared expert width; 0 = no shared expert, else % 128 == 0 */
  int32_t R;            /* logical ranks; expert e lives on rank e / (E/R), token t is sent by
                           rank t / (T/R); R <= 64 */
  float route_scale;    /* factor applied to the renormalised gate weights */
  int32_t act_dtype;    /* dispatched activations: MOE_BF16, MOE_FP8_E4M3 or MOE_FP8_E4M3_POW2 */
  int32_t w_dtype;      /* expert weights: must equal act_dtype */
} moe_cfg;

/* Buffer sizes the caller allocates for a configuration. */
typedef struct moe_sizes {
  int64_t recv_rows;        /* R * R * cap rows in the receive buffer */
  int32_t cap;              /* rows per (destination rank, source rank) segment:
                               (T/R) * min(k, E/R), the most one source can send one rank */
  size_t recv_bytes;        /* recv: [R][R][cap][d], bf16 (2 B) or e4m3 (1 B) elements */
  size_t recv_scale_bytes;  /* e4m3 only: recv_scales fp32, block-major [d/128][recv_rows]
                               (scale of block b of row j at b * recv_rows + j); else 0 */
  size_t ebuf_bytes;        /* ebuf: expert outputs, bf16 [R][R][cap][d] (same rows as recv) */
  size_t ws_bytes;          /* ws: scratch workspace (status word, router partials, tile
                               schedule, SwiGLU intermediates) */
} moe_sizes;

/* Expert weights, K-major (the reduction dimension is contiguous).
 *  w13  [E][2*d_ff][d]: rows 0..d_ff-1 are the gate projection, d_ff..2*d_ff-1 the up one.
 *  w2   [E][d][d_ff]:   down projection.
 *  ws13 [2*d_ff_shared][d], ws2 [d][d_ff_shared]: the shared expert (NULL if none).
 *  e4m3 weights carry one fp32 scale per 128x128 block: w13_scales [E][2*d_ff/128][d/128],
 *  w2_scales [E][d/128][d_ff/128], ws13_scales [2*d_ff_shared/128][d/128],
 *  ws2_scales [d/128][d_ff_shared/128]; all scale pointers are NULL for bf16. */
typedef struct moe_weights {
  const void* w13;
  const float* w13_scales;
  const void* w2;
  const float* w2_scales;
  const void* ws13;
  const float* ws13_scales;
  const void* ws2;
  const float* ws2_scales;
} moe_weights;

/* Checks a configuration. Returns MOE_OK, MOE_ERR_INVALID_ARG or MOE_ERR_UNSUPPORTED. */
int moe_validate(const moe_cfg* cfg);

/* Fills *out with the buffer sizes for cfg. Same return codes as moe_validate. */
int moe_query_sizes(const moe_cfg* cfg, moe_sizes* out);

/* Router ("Mixture-of-experts serving", paragraphs 1 and 3; "Serving Mixture-of-Experts",
 * Expert Parallelism Mechanics, router step). For every token t:
 *   z[e] = x[t] . w_gate[e] in fp32, summed in a fixed order: d in 16 equal chunks, each a
 *          sequential fused multiply-add chain, the 16 partials added by a pairwise tree;
 *   s[e] = 1 / (1 + exp(-z[e])) (exp by Cody-Waite reduction and a degree-7 Taylor series);
 *   v[e] = s[e] + bias[e]   (the bias steers selection only);
 *   group score = sum of the two largest v in the group; the topk_group best groups are kept;
 *   the k best experts of the kept groups by v are chosen (ties: lower index first);
 *   topk_w[t][i] = s[e_i] / (s[e_0] + ... + s[e_{k-1}]) * route_scale.
 * x bf16 [T][d]; w_gate fp32 [E][d]; bias fp32 [E]; outputs topk_idx int32 [T][k] in
 * selection order and topk_w fp32 [T][k]. ws: workspace of moe_sizes.ws_bytes. */
int moe_route(const moe_cfg* cfg, const void* x, const float* w_gate, const float* bias,
              int32_t* topk_idx, float* topk_w, void* ws, cudaStream_t stream);

/* The router of moe_route for callers that cannot give the library any device memory beyond
 * their inputs and outputs: a plugin inside another framework with no access to its
 * allocator, a deployment whose device memory is fully planned at start-up, or a hot path that
 * must not enter the driver allocator (cudaMalloc/cudaFree can synchronise the device). It
 * needs no ws: its scratch (16 partial dot products per token and expert) is a fixed 8 MiB
 * device array inside the library, which every device that loads the library holds until the
 * process exits. The pages have no counterpart to this entry point; it exists for such
 * callers only. Arguments and results are those of moe_route. Limits and behaviour:
 *  - returns MOE_ERR_UNSUPPORTED when 16 * T * E exceeds 2^21 floats (T*E > 131072, e.g. more
 *    than 512 tokens at 256 experts); nothing is enqueued then;
 *  - the first call in each device context looks up the array's device address with that
 *    device current (cudaGetSymbolAddress) and caches it under the context's ID; make that
 *    first call before any stream capture (a context made after a device reset looks it up
 *    again on its own first call);
 *  - it allocates nothing (no cudaMalloc, no cudaFree, no allocating library call);
 *  - every call shares the array and leaves its contents behind; each call writes every entry
 *    it reads, so nothing needs clearing, but calls whose kernels overlap on the GPU (other
 *    streams, other host threads on the same device) race on it: serialise them. */
int moe_route_noalloc(const moe_cfg* cfg, const void* x, const float* w_gate, const float* bias,
                      int32_t* topk_idx, float* topk_w, cudaStream_t stream);

/* Dispatch ("Serving Mixture-of-Experts", Expert Parallelism Mechanics, dispatch step;
 * "One-Sided Expert-Parallel All-to-All...", abstract; "Serving Mixture-of-Experts", DeepEP,
 * FP8 dispatch and fixed-size buffers). Each logical source rank s (tokens s*T/R ..) counts
 * its rows per expert, takes exclusive sums of those counts inside each destination rank, and
 * writes one row per (token, chosen expert) into segment (r = rank(e), s) of the receive
 * buffer: row (r*R + s)*cap + [sum of counts[s][e'] for e' on rank r, e' < e] + [number of
 * earlier tokens of s that chose e]. No count is exchanged before the rows are written.
 * bf16: recv[row] = x[t]. e4m3: x[t] is quantised once per 128-column block (scale =
 * amax/448, or 1 if amax is 0; code = e4m3(x/scale), nearest even, saturating) and written to
 * each of its rows; the block scales are block-major, recv_scales[b * recv_rows + row], so the
 * expert GEMMs read one K block's scales for consecutive rows from consecutive addresses.
 * Inputs x bf16 [T][d], topk_idx int32 [T][k] (entries in [0, E), distinct per token).
 * Outputs recv (see moe_sizes), recv_scales (e4m3 only, else NULL), counts int32 [R][E],
 * row_of int32 [T][k] (receive row of each choice), src_tok int32 [recv_rows] (token of each
 * row, -1 for empty rows; NULL to skip). Receive rows that get no token are not written.
 * status: NULL, or a device uint32 (for instance the workspace's status word: pass ws) into
 * which MOE_DEV_BOUNDS is OR-ed when topk_idx breaks its contract. A choice whose expert is
 * outside [0, E), or repeats an earlier choice of the same token, is skipped: its row_of is
 * -1, it is not counted, and nothing is written for it. With distinct experts no segment can
 * overflow; every receive row written lies inside recv. moe_route never produces either. */
int moe_dispatch(const moe_cfg* cfg, const void* x, const int32_t* topk_idx, void* recv,
                 float* recv_scales, int32_t* counts, int32_t* row_of, int32_t* src_tok,
                 uint32_t* status, cudaStream_t stream);

/* Expert FFNs ("Serving Mixture-of-Experts", Expert Parallelism Mechanics, expert compute: a
 * grouped GEMM over the rows each expert received; Hot-Expert Skew section and
 * "Mixture-of-experts serving" paragraph 1: the always-on shared expert). For every filled
 * receive row of expert e, read in place from recv:
 *   h = silu(row . Wgate_e^T) * (row . Wup_e^T), rounded to the activation format
 *       (e4m3: re-quantised per 128 columns like the dispatch);
 *   ebuf[row] = bf16(h . Wdown_e^T).
 * The shared expert does the same for every token of x: shared_out[t] (bf16 [T][d]).
 * counts: the dispatch's counts [R][E] (the only metadata; rows are located from it).
 * x: bf16 [T][d], the shared expert's input (NULL when d_ff_shared == 0). For e4m3 the shared
 * input is quantised here with the dispatch's rule. Rows of ebuf that hold no token are not
 * written. ws: workspace (holds the tile schedule and the SwiGLU intermediates). The two
 * GEMMs follow this call's own schedule kernels with programmatic launches (see moe_layer). */
int moe_expert_ffn(const moe_cfg* cfg, const void* recv, const float* recv_scales,
                   const int32_t* counts, const void* x, const moe_weights* w, void* ebuf,
                   void* shared_out, void* ws, cudaStream_t stream);

/* Combine ("Serving Mixture-of-Experts", Expert Parallelism Mechanics, combine step: the k
 * partial results of a token weighted-summed by its gate weights; DeepEP section: BF16
 * combine). y[t] = bf16( sum_i topk_w[t][i] * ebuf[row_of[t][i]] + shared_out[t] ), summed in
 * fp32 in selection order. ebuf bf16 [recv_rows][d]; row_of int32 [T][k]; topk_w fp32
 * [T][k]; shared_out bf16 [T][d] or NULL; y bf16 [T][d]. Passing the receive buffer as ebuf
 * (bf16) gives route_scale * x: the identity-expert check of the dispatch/combine pair.
 * Negative entries of row_of are skipped (a choice the dispatch skipped). Entries at or past
 * recv_rows are skipped too and reported: MOE_DEV_BOUNDS is OR-ed into status (NULL, or a
 * device uint32 such as the workspace's status word). Nothing outside ebuf is read.
 * moe_dispatch's row_of holds only valid rows and -1. */
int moe_combine(const moe_cfg* cfg, const void* ebuf, const int32_t* row_of,
                const float* topk_w, const void* shared_out, void* y, uint32_t* status,
                cudaStream_t stream);

/* The whole layer on one stream: moe_route, moe_dispatch, moe_expert_ffn, moe_combine.
 * Buffers as in those calls (src_tok is not produced). events: NULL, or MOE_LAYER_EVENTS
 * created events that are recorded on `stream` before the router, after the router, after
 * the dispatch, after the FFN set-up (schedule and shared-input quantisation), after the
 * gate/up GEMM, after the down GEMM, and after the combine.
 * With events == NULL every kernel after the first is launched with programmatic stream
 * serialisation: it may become resident while the previous kernel runs, and waits for that
 * kernel to finish before it touches memory. The first kernel (the router's) starts after the
 * work already on `stream`, as any launch. With events, the stages are launched one after
 * another so that the events time them. With a shared expert, the router's selection kernel
 * also starts prefetching w->ws13 into L2 (reads only; the gate/up GEMM reads it first). */
int moe_layer(const moe_cfg* cfg, const void* x, const float* w_gate, const float* bias,
              const moe_weights* w, int32_t* topk_idx, float* topk_w, void* recv,
              float* recv_scales, int32_t* counts, int32_t* row_of, void* ebuf,
              void* shared_out, void* y, void* ws, cudaStream_t stream,
              const cudaEvent_t* events);

/* ---------------------------------------------------------------------------------------
 * Variants of the layer ("next" steps of the method, each optional)
 * ------------------------------------------------------------------------------------- */

/* Gather mode. The dispatch writes only the indices (counts, row_of and the token of each
 * receive row); the gate/up GEMM reads each routed row straight from x by token instead of
 * from a receive-buffer copy, so the copy pass and its Tk*d bytes of writes and reads are
 * skipped. The grouped GEMMs reading pushed rows in place is the design of "One-Sided
 * Expert-Parallel All-to-All ..." (abstract); "DeepSeek MoE Serving: Where Expert-Parallel
 * All-to-All Time Goes" (groundy) counts the extra pass of a two-sided scheme as HBM traffic.
 * On one GPU the source rank's own x is the pushed buffer, read in place. e4m3: x is
 * quantised once per token (not once per (token, expert) row) with the dispatch's rule. The
 * expert outputs still land in ebuf at the receive rows, so the combine is unchanged and every
 * output equals moe_layer's. recv and recv_scales are not used (may be NULL). */
#define MOE_OPT_GATHER_X 1u
/* Shared expert on a second stream ("Serving Mixture-of-Experts", Hot-Expert Skew: the shared
 * expert's FFN needs no all-to-all, so it is free work to overlap with the dispatch; DeepEP
 * section: hook-based overlap). Its GEMMs depend only on x: they are enqueued on side_stream
 * after fork_event (recorded on `stream` at the start of the layer), limited to side_ctas CTAs
 * (one per SM, leaving the other SMs to the router and dispatch), and the combine waits on
 * join_event (recorded on side_stream after them). On one GPU this partitions the SMs between
 * the two streams. The events are created by the caller (cudaEventDisableTiming is enough). */
#define MOE_OPT_SHARED_SIDE_STREAM 2u
/* Fused expert stage (bf16 only): the gate/up GEMM, the down GEMM and the combine run in one
 * persistent cooperative launch ("DeepSeek MoE Serving: Where Expert-Parallel All-to-All Time
 * Goes" (groundy), regimes table and the paragraph after it: a fused MoE kernel against
 * separate kernels). A down unit starts as soon as the gate/up units of its own token tile
 * have published their rows (device-side counters in ws, every wait bounded), so SMs that run
 * out of gate/up units do not idle until the whole stage ends; the combine follows in the same
 * launch. Not with MOE_OPT_SHARED_SIDE_STREAM (MOE_ERR_INVALID_ARG) or e4m3
 * (MOE_ERR_UNSUPPORTED). Stage events 4..6 are all recorded after the launch. */
#define MOE_OPT_FUSED_FFN 4u

/* Redundant experts ("Serving Mixture-of-Experts", Hot-Expert Skew: place extra copies of the
 * busiest experts on under-loaded ranks and let the dispatch split their tokens across the
 * copies; exercise 5: each copy takes an equal share of its expert's load, copies assigned
 * largest first to the least-loaded rank). Each of the R logical ranks has slots_per_rank
 * expert slots, G = R * slots_per_rank >= E in all; slot p lives on rank p / slots_per_rank.
 * The dispatch sends source s's j-th row of expert e (in token order) to copy
 * (j + s) mod n_copies[e]: every source splits its own rows of an expert evenly over the
 * copies without exchanging counts. All arrays are DEVICE int32 arrays owned by the caller,
 * normally filled from moe_place_experts:
 *  slot_expert [G]: the expert each slot holds; n_copies [E]: copies of each expert (>= 1);
 *  copy_slot [E][max_copies]: the slots of each expert's copies in ascending order.
 * With a placement the receive layout and counts are over the G slots (counts [R][G],
 * cap = (T/R) * min(k, slots_per_rank); moe_query_sizes_placed gives the sizes). The expert
 * GEMMs take the rows of all copies of an expert through its weights together (one GPU holds
 * one set of weights per expert), so the output equals moe_layer's bit for bit. */
typedef struct moe_placement {
  int32_t slots_per_rank;
  int32_t max_copies;
  const int32_t* slot_expert;
  const int32_t* n_copies;
  const int32_t* copy_slot;
} moe_placement;

typedef struct moe_layer_opts {
  uint32_t flags;           /* MOE_OPT_* bits; 0 = moe_layer */
  cudaStream_t side_stream; /* MOE_OPT_SHARED_SIDE_STREAM: the shared expert's stream */
  cudaEvent_t fork_event;   /* recorded on `stream`, waited on by side_stream */
  cudaEvent_t join_event;   /* recorded on side_stream, waited on by `stream` */
  int32_t side_ctas;        /* CTAs of each shared-expert GEMM; 0 = 16 */
  const moe_placement* placement; /* NULL, or redundant experts placed on slots (above) */
} moe_layer_opts;

/* Placement of E experts on R ranks of slots_per_rank slots from estimated loads (host
 * function, no GPU; load: host double [E], e.g. a moving average of past counts). The
 * R*slots_per_rank - E spare slots take one more copy at a time of the expert with the largest
 * load per copy (ties: lower expert). Each copy carries load/copies; copies are placed largest
 * first (ties: lower expert, then lower copy) on the least-loaded rank that has a free slot
 * (ties: lower rank); a rank's slots are ordered by (expert, copy). Outputs (host int32):
 * slot_expert [R*slots_per_rank], n_copies [E], copy_slot [E][max_copies] (-1 past a copy
 * count). Returns MOE_ERR_INVALID_ARG for a NULL pointer, non-positive sizes, a negative or
 * non-finite load, R*slots_per_rank < E, or an expert needing more than max_copies copies. */
int moe_place_experts(int32_t E, int32_t R, int32_t slots_per_rank, const double* load,
                      int32_t max_copies, int32_t* slot_expert, int32_t* n_copies,
                      int32_t* copy_slot);

/* moe_query_sizes for a layer whose experts are placed on R*slots_per_rank slots. */
int moe_query_sizes_placed(const moe_cfg* cfg, int32_t slots_per_rank, moe_sizes* out);

/* moe_layer with the variants selected by opts (NULL = moe_layer). Arguments as in moe_layer;
 * with MOE_OPT_GATHER_X, recv and recv_scales may be NULL. With MOE_OPT_SHARED_SIDE_STREAM and
 * a shared expert, side_stream, fork_event and join_event must be valid (else
 * MOE_ERR_INVALID_ARG); stage events are recorded on `stream` only, so the FFN stages then
 * time the routed experts alone. With a placement, recv, counts, ebuf and ws are sized by
 * moe_query_sizes_placed and counts is [R][G] over the slots; a slot whose expert lies outside
 * [0, E) is reported (MOE_DEV_BOUNDS) and computed with expert 0's weights. The layer output
 * y is moe_layer's in every mode, bit for bit. */
int moe_layer_ex(const moe_cfg* cfg, const moe_layer_opts* opts, const void* x,
                 const float* w_gate, const float* bias, const moe_weights* w, int32_t* topk_idx,
                 float* topk_w, void* recv, float* recv_scales, int32_t* counts, int32_t* row_of,
                 void* ebuf, void* shared_out, void* y, void* ws, cudaStream_t stream,
                 const cudaEvent_t* events);

/* The index pass of moe_dispatch alone (gather mode): counts, row_of and src_tok exactly as
 * moe_dispatch writes them (src_tok required here; receive rows that get no token hold -1),
 * with no payload copied. status as in moe_dispatch. */
int moe_dispatch_index(const moe_cfg* cfg, const int32_t* topk_idx, int32_t* counts,
                       int32_t* row_of, int32_t* src_tok, uint32_t* status,
                       cudaStream_t stream);

/* moe_expert_ffn in gather mode: the routed rows are read from x by token through src_tok
 * (from moe_dispatch_index) instead of from a receive buffer. x: bf16 [T][d], required. The
 * outputs (ebuf at the receive rows, shared_out) equal moe_expert_ffn's. */
int moe_expert_ffn_gather(const moe_cfg* cfg, const void* x, const int32_t* counts,
                          const int32_t* src_tok, const moe_weights* w, void* ebuf,
                          void* shared_out, void* ws, cudaStream_t stream);

/* ---------------------------------------------------------------------------------------
 * Training of the expert path
 *
 * The gradients of the expert stage and what they need from the forward pass. One training step
 * of the layer's experts, with the dispatch of a one-rank configuration (R = 1: expert e's rows
 * are contiguous, in expert order, counts [E]):
 *   forward : moe_route, moe_dispatch -> moe_grouped_mm (gate/up) -> moe_swiglu_save
 *             -> moe_grouped_mm (down) -> moe_combine;   moe_act_save keeps x
 *   backward: moe_combine_grad -> moe_grouped_mm_dx, moe_grouped_mm_dw (down)
 *             -> moe_swiglu_grad -> moe_grouped_mm_dx (gate/up)
 *             -> moe_act_load (x's rows) -> moe_grouped_mm_dw (gate/up)
 *             -> moe_combine with weights of one (dx: the dispatch's gradient)
 * The pages cover inference only and have no counterpart to these calls.
 *
 * An output (the workspace of a grouped product too) may not overlap an input or another output:
 * MOE_ERR_INVALID_ARG. Two may be the very array they take the place of: moe_swiglu_grad's a that
 * of da, moe_combine_grad's dtopk_w that of topk_w.
 * ------------------------------------------------------------------------------------- */

/* Shape of one grouped product. The row tensors hold the rows of the E groups one group after
 * another: group e owns rows [s_e, s_e + counts[e]), s_e = counts[0] + ... + counts[e-1]. rows, n
 * and k are at most 2^31 - 513. */
typedef struct moe_group_cfg {
  int32_t rows;  /* rows of the row tensors, >= 0; the groups own the first sum(counts) of them */
  int32_t E;     /* groups (experts), 1 <= E <= 1024 */
  int32_t n;     /* rows of each group's weight matrix; n % 8 == 0 */
  int32_t k;     /* its columns; k % 8 == 0 */
} moe_group_cfg;

/* Bytes of the workspace that the grouped products of this shape take. The first word of the
 * workspace is its status word (moe_clear_status, moe_read_status); the caller zeroes the
 * workspace once, before its first use, and every call leaves it ready for the next (after a
 * call that reported MOE_DEV_TIMEOUT, zero it again). Calls that
 * may overlap on the GPU need workspaces of their own. MOE_ERR_INVALID_ARG for a negative or
 * zero size, MOE_ERR_UNSUPPORTED for n or k not a multiple of 8, E > 1024 or a size past
 * 2^31 - 513. */
int moe_grouped_query(const moe_group_cfg* cfg, size_t* ws_bytes);

/* Matrix products grouped by expert, rows of any number per group (0 included). bf16 operands,
 * sums in fp32. counts: int32 [E] on the device (as moe_dispatch writes them for R = 1), read on
 * the device, so no call waits for them. A negative count, or counts that pass `rows` in all,
 * are reported (MOE_DEV_BOUNDS) and cut to what fits. Rows that no group owns are neither read
 * into a result nor written.
 *   forward:            y[r]  = bf16( x[r] . W_e^T )        x [rows][k], w [E][n][k], y [rows][n]
 *   gradient of rows:   dx[r] = bf16( dy[r] . W_e )         dy [rows][n], dx [rows][k]
 *   gradient of W:      dW_e  = sum over the group's rows of dy[r]^T x[r]         dw [E][n][k]
 * dw_dtype: MOE_BF16 or MOE_F32. accumulate (MOE_F32 only, else MOE_ERR_INVALID_ARG): dW_e is
 * added to dw instead of replacing it. An empty group's dW_e is 0. The results do not depend on
 * the order in which the GPU runs the work (no floating-point atomics). With rows == 0 the row
 * tensors may be NULL, and counts are not read. */
#define MOE_F32 3 /* dw_dtype, the residual stream of the norms, gradients of the optimiser */
int moe_grouped_mm(const moe_group_cfg* cfg, const void* x, const int32_t* counts, const void* w,
                   void* y, void* ws, cudaStream_t stream);
int moe_grouped_mm_dx(const moe_group_cfg* cfg, const void* dy, const int32_t* counts,
                      const void* w, void* dx, void* ws, cudaStream_t stream);
int moe_grouped_mm_dw(const moe_group_cfg* cfg, const void* dy, const void* x,
                      const int32_t* counts, void* dw, int32_t dw_dtype, int32_t accumulate,
                      void* ws, cudaStream_t stream);

/* Activation checkpoints in 8 bits: bf16 rows kept for the backward pass as e4m3 codes with one
 * fp32 scale per 128 columns, by the dispatch's rule (scale = amax/448, or 1 if amax is 0; code
 * = e4m3(x/scale), nearest even, saturating; the amax is over the block's numbers). Scales are
 * block-major: the scale of block b of row r at scales[b * rows + r]. A NaN stays a NaN; an
 * infinity makes its block read back as NaN. Here and in the two calls below, rows times columns
 * (d or f) at or past 2^37 is MOE_ERR_UNSUPPORTED.
 * moe_act_save: x bf16 [rows][d] -> q [rows][d] bytes, scales [d/128][rows]. d % 128 == 0.
 * moe_act_load: out[i] = bf16(code * scale) of saved row index[i] (index int32 [rows], NULL: row
 *   i), out bf16 [rows][d]; src_rows: the saved rows. An index of -1 gives a row of zeros; any
 *   other index outside [0, src_rows) does too and is reported (MOE_DEV_BOUNDS in status, NULL
 *   or a device uint32). With the token of each expert row as the index (src_tok of
 *   moe_dispatch), x is kept once per token, not once per expert row. */
int moe_act_save(int32_t rows, int32_t d, const void* x, void* q, float* scales,
                 cudaStream_t stream);
int moe_act_load(int32_t rows, int32_t src_rows, int32_t d, const void* q, const float* scales,
                 const int32_t* index, void* out, uint32_t* status, cudaStream_t stream);

/* SwiGLU of the gate/up product, keeping its input in 8 bits. gu bf16 [rows][2f] (gate, then
 * up), f % 128 == 0: a = bf16(silu(g) * u) [rows][f] from the bf16 values; q [rows][2f] and
 * scales [2f/128][rows] as moe_act_save(gu). */
int moe_swiglu_save(int32_t rows, int32_t f, const void* gu, void* a, void* q, float* scales,
                    cudaStream_t stream);

/* Gradient of that SwiGLU from the saved codes, g and u being code * scale, s = 1/(1+exp(-g)):
 *   dgu = bf16 of [ da u s (1 + g (1 - s)) | da g s ]   [rows][2f];  da bf16 [rows][f]
 *   a   = bf16(g s u) [rows][f], the down product's input again (NULL: not wanted). */
int moe_swiglu_grad(int32_t rows, int32_t f, const void* q, const float* scales, const void* da,
                    void* dgu, void* a, cudaStream_t stream);

/* Gradient of moe_combine. dy bf16 [T][d]; row_of int32 [T][k] and topk_w fp32 [T][k] as given to
 * the combine; ebuf bf16 [rows][d] its expert rows:
 *   debuf[row_of[t][i]] = bf16(topk_w[t][i] * dy[t]);  dtopk_w[t][i] = dy[t] . ebuf[row_of[t][i]]
 * (summed in fp32 in a fixed order). No two choices may name one row (the dispatch gives each its
 * own). Rows of debuf that no choice names are not written. A
 * negative row_of is a choice that the dispatch skipped: its dtopk_w is 0. One at or past rows is
 * treated so too and reported (MOE_DEV_BOUNDS in status, NULL or a device uint32). The shared
 * expert's rows have dy itself as gradient. d % 128 == 0, 1 <= k <= 32, T * k < 2^31. */
int moe_combine_grad(int32_t T, int32_t k, int32_t d, int32_t rows, const void* ebuf,
                     const int32_t* row_of, const float* topk_w, const void* dy, void* debuf,
                     float* dtopk_w, uint32_t* status, cudaStream_t stream);

/* ---------------------------------------------------------------------------------------
 * The rest of a training step of an MoE block: the norms around the layer, the router's gradient,
 * the optimiser. A block is
 *   n = norm(x) w  ->  y = moe_layer(n)  ->  h = res x + out gate norm(y) w_post (-> next n)
 * The pages cover neither training nor the norms and have no counterpart to these calls. As in the
 * section above, an output may not overlap an input or another output (MOE_ERR_INVALID_ARG) except
 * where a call says that it may take an input's place (the very array).
 * ------------------------------------------------------------------------------------- */

#define MOE_GATE_NONE 0
#define MOE_GATE_CHANNEL 1   /* fp32 [d]: one factor a column (a learned layer scale) */
#define MOE_GATE_TOKEN 2     /* fp32 [rows]: one factor a row */
#define MOE_GATE_ELEMENT 3   /* bf16 [rows][d] */

typedef struct moe_norm_cfg {
  int32_t rows;           /* >= 0 */
  int32_t d;              /* d % 8 == 0, d <= 16384; rows * d < 2^37 */
  float eps;              /* finite, >= 0 (0: a row of zeros has no norm, and gives NaN) */
  float res_scale;        /* res: factor of the residual stream (norm_out) */
  float out_scale;        /* out: factor of the block's gated output (norm_out) */
  int32_t stream_dtype;   /* MOE_BF16 or MOE_F32: type of the residual stream (x, h, dh, dx) */
  int32_t gate;           /* MOE_GATE_* (norm_out) */
} moe_norm_cfg;

/* RMS norm before a block: r = 1/sqrt(mean_j x_j^2 + eps) of each row, n = bf16(x r w).
 * x [rows][d] of the stream's type, w fp32 [d], n bf16 [rows][d] (may take the place of a bf16 x),
 * rstd fp32 [rows]: r, kept for the gradient (NULL: not wanted). Squares and sums in fp32 here and
 * below: values past 1e19 leave its range, and so do, with an eps of 0 or near it, rows of values that
 * are all below 1e-18. */
int moe_norm_in(const moe_norm_cfg* cfg, const void* x, const float* w, void* n, float* rstd,
                cudaStream_t stream);

/* Its gradient: dx = dres + r (dn w - xh mean(dn w xh)), xh = x r; dw = sum over rows of dn xh
 * (fp32 [d]; accumulate: added to dw; NULL: not wanted). dn bf16; dres (the gradient that reaches x
 * by the residual, NULL: none) and dx of the stream's type; dx may take dres's place. ws: scratch
 * of moe_norm_query bytes (no initial value; calls that may overlap on the GPU need their own). */
int moe_norm_in_grad(const moe_norm_cfg* cfg, const void* dn, const void* x, const float* w,
                     const float* rstd, const void* dres, void* dx, float* dw, int32_t accumulate,
                     void* ws, cudaStream_t stream);

/* Norm after a block, gate, residual and the norm before the next block in one pass:
 *   s = y r_y w_post (w_post NULL: s = y)      r_y as above, from y
 *   h = res x + out gate s                     in fp32, stored in the stream's type
 *   n = bf16(h r_h w_next) (w_next NULL: none) r_h and n from h before its rounding
 * y bf16 [rows][d], the block's output; x the residual stream; gate by cfg->gate (NULL for NONE);
 * h may take x's place, n that of y. rstd_y, rstd_h fp32 [rows] (NULL: not wanted). */
int moe_norm_out(const moe_norm_cfg* cfg, const void* y, const void* x, const float* w_post,
                 const void* gate, const float* w_next, void* h, void* n, float* rstd_y,
                 float* rstd_h, cudaStream_t stream);

/* Its gradient, from dh (NULL: none) and dn (with w_next), from y (needed with w_post or a gate),
 * from h as stored and rstd_h (with w_next), and rstd_y (with w_post). With hh = h r_h, yh = y r_y:
 *   G  = dh + r_h (dn w_next - hh mean(dn w_next hh))
 *   dx = res G                        ds = out gate G        dgate = out G s, summed to the
 *   dy = r_y (ds w_post - yh mean(ds w_post yh)) (or ds)     gate's shape, in the gate's type
 *   dw_post = sum over rows of ds yh  dw_next = sum over rows of dn hh
 * dx (may take dh's place), dgate, dw_post, dw_next: NULL where not wanted; dy may take dn's place.
 * accumulate: dw_post, dw_next and a CHANNEL gate's dgate are added to. The sums do not depend on
 * the order in which the GPU runs the work. ws as in moe_norm_in_grad. Without rows the gate, too,
 * may be NULL, and the sums are 0. */
int moe_norm_out_grad(const moe_norm_cfg* cfg, const void* dh, const void* dn, const void* y,
                      const void* h, const float* w_post, const void* gate, const float* w_next,
                      const float* rstd_y, const float* rstd_h, void* dx, void* dy, void* dgate,
                      float* dw_post, float* dw_next, int32_t accumulate, void* ws,
                      cudaStream_t stream);

/* Bytes of the scratch of the two gradients. MOE_ERR_INVALID_ARG for rows < 0 or d < 1,
 * MOE_ERR_UNSUPPORTED for a d or a size that the calls do not take. */
int moe_norm_query(int32_t rows, int32_t d, size_t* ws_bytes);

/* moe_route that also keeps the raw sigmoid scores of the chosen experts, topk_s fp32 [T][k], for
 * moe_route_grad. topk_idx and topk_w are moe_route's, bit for bit. */
int moe_route_save(const moe_cfg* cfg, const void* x, const float* w_gate, const float* bias,
                   int32_t* topk_idx, float* topk_w, float* topk_s, void* ws,
                   cudaStream_t stream);

/* Gradient of the router, from that of its weights (dtopk_w fp32 [T][k], as moe_combine_grad gives
 * it). The choice has no gradient (nor has the bias, which steers it alone). With s = topk_s and
 * p_i = s_i / (s_0 + ... + s_{k-1}), so that topk_w_i = route_scale p_i:
 *   dz_i = route_scale p_i (1 - s_i) (dtopk_w_i - sum_j p_j dtopk_w_j)
 *   dx[t] = bf16(dx_in[t] + sum_i dz_i w_gate[e_i])          e_i = topk_idx[t][i]
 *   dw_gate[e] = sum of dz x[t] over the choices of e        fp32 [E][d]; accumulate: added to
 * x, dx_in (NULL: none), dx bf16 [T][d]; dx may take dx_in's place. Sums in fp32 in a fixed order.
 * A choice outside [0, E) gets no gradient and gives none (its p and its dtopk_w, which
 * moe_combine_grad sets to 0, count in the sums over j) and is reported
 * (MOE_DEV_BOUNDS in the first word of ws; -1, a choice that was dropped, is not reported). Of cfg,
 * T, d, E, k and route_scale count; d <= 65536, T * d < 2^37 and T * k <= 2^31 - 2048 (else
 * MOE_ERR_UNSUPPORTED). ws:
 * moe_route_grad_query bytes; zero its first word once. Calls that may overlap on the GPU need
 * workspaces of their own. */
int moe_route_grad(const moe_cfg* cfg, const void* x, const float* w_gate, const int32_t* topk_idx,
                   const float* topk_s, const float* dtopk_w, const void* dx_in, void* dx,
                   float* dw_gate, int32_t accumulate, void* ws, cudaStream_t stream);
int moe_route_grad_query(const moe_cfg* cfg, size_t* ws_bytes);

/* One tensor of an optimiser's step (an entry of a HOST array; the pointers are device pointers).
 * With moments in 32 bits m and v are fp32 [n], m_scale and v_scale are NULL. In 8 bits m and v are
 * e4m3 codes [n] of m and of sqrt(v), each block of 128 consecutive elements with an fp32 scale
 * (m_scale, v_scale [ceil(n/128)]). Moments and scales start at zero. */
typedef struct moe_adam_tensor {
  float* p;             /* parameters, fp32 [n] */
  const void* g;        /* their gradient, fp32 or bf16 [n] */
  void* w;              /* bf16 copy of p that the step refreshes; NULL: none */
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;            /* elements, 0 <= n < 2^39 */
  float weight_decay;   /* finite, >= 0 */
  uint32_t seed;        /* 8 bits: of the tensor's random numbers; another one for each tensor */
  int32_t g_dtype;      /* MOE_F32 or MOE_BF16 */
  int32_t reserved;     /* 0 */
} moe_adam_tensor;

typedef struct moe_adam_cfg {
  double lr;            /* finite, >= 0 */
  double beta1, beta2;  /* in [0, 1) */
  double eps;           /* > 0, in fp32 too */
  double max_norm;      /* largest norm of all gradients; 0: they are not clipped */
  const float* lr_dev;  /* NULL, or a device scalar that is read in lr's place (for a captured step
                           whose rate changes between replays) */
  int32_t state_bits;   /* 32 or 8 */
  int32_t reserved;     /* 0 */
} moe_adam_cfg;

/* Tensors a call takes at most. A step over more of them is made of several calls, all but the last
 * with `more` set. */
#define MOE_ADAM_TENSORS 256

/* AdamW (I. Loshchilov and F. Hutter, "Decoupled weight decay regularization", 2019), step t, over
 * n tensors in one launch:
 *   g' = g min(1, max_norm / *norm)          (max_norm 0 or norm NULL: g' = g)
 *   m  = b1 m + (1 - b1) g'                  v = b2 v + (1 - b2) g'^2
 *   p  = p - lr weight_decay p - lr/(1 - b1^t) m / (sqrt(v/(1 - b2^t)) + eps);   w = bf16(p)
 * p moves by the new moments in fp32, before they are put into 8 bits. There, q = |m| / scale or
 * q = sqrt(v) / scale (scale = amax * fp32(1/448) of the block; max_norm / norm is max_norm *
 * (1/norm); IEEE operations, each of these and of m and v above rounded by itself) is rounded to a
 * neighbouring code at random, by 16 random bits an element from (seed, t, element), with odds that
 * keep the mean of m and of v: with nearest rounding a v with b2 near 1 would not move. A code of v
 * is never 0 where v is not. A block whose scale would be below 2^-126 (of m: amax below 5e-36; a
 * root of v is 0 or above 1e-23) has scale 1 and codes 0.
 * A NaN or an infinity in m or v spoils its block: it becomes the block's scale.
 * state: moe_adam_query bytes, zeroed once (step 0); it holds the status word, t, the bias
 * corrections and the partial sums of moe_grad_norm. The last call of a step advances t.
 * norm: NULL, or the device scalar of moe_grad_norm (needed with max_norm > 0). Where it is not
 * finite the step is left out (nothing is written, t stays) and MOE_DEV_NONFINITE is reported.
 * Results do not depend on the order in which the GPU runs the work. p, w, m, v and the scales are
 * read and written in place; no two of the call's arrays may overlap. */
int moe_adamw(const moe_adam_cfg* cfg, const moe_adam_tensor* tensors, int32_t n, int32_t more,
              void* state, const float* norm, cudaStream_t stream);

/* norm = sqrt of the sum of all g^2 (device fp32 scalar; squares in fp32, so that a gradient past
 * 1e19 counts as infinite and one below 1e-23 as 0). Of the tensors, g, g_dtype and n count. With
 * `more` the sum goes on in the next call and norm is not written (a norm that was broken off is
 * ended by a call with n = 0). Calls that may overlap on the GPU need states of their own, here and
 * in moe_adamw. */
int moe_grad_norm(const moe_adam_tensor* tensors, int32_t n, int32_t more, void* state,
                  float* norm, cudaStream_t stream);

/* Bytes of the state. Its layout, for saving and loading: uint32 status, uint32 (scratch, 0), int64
 * t, double 1 - b1^t, double 1 - b2^t, then scratch that is 0 between steps or written before it is
 * read. */
int moe_adam_query(size_t* state_bytes);

/* Sets the device status word in ws to 0 (enqueued on stream). */
int moe_clear_status(void* ws, cudaStream_t stream);

/* Synchronises `stream`, then copies the device status word of ws into *status (MOE_DEV_*
 * bits). This is the one call that blocks the host. */
int moe_read_status(const void* ws, uint32_t* status, cudaStream_t stream);

/* Diagnostic of the device-side failure handling (the pages have no counterpart; it serves
 * callers and tests that must see a kernel give up instead of hang). Launches one CTA in which
 * one thread waits on a barrier that nothing ever completes, bounded by limit_ns, while a
 * second thread waits on another such barrier with a limit three times as long. When the first
 * wait runs out it ORs MOE_DEV_TIMEOUT into the status word of ws and raises the CTA's abort
 * flag, on which the second wait returns at once; the kernel then ends (after about limit_ns,
 * well before 3 x limit_ns) and the context stays usable. ws: any workspace of this library
 * (only its status word is written). limit_ns: 1 us .. 10 s, else MOE_ERR_INVALID_ARG. */
int moe_selftest_wait(void* ws, int64_t limit_ns, cudaStream_t stream);

/* Static name of a return code. */
const char* moe_strerror(int code);

/* MOE_ABI_VERSION of the library. */
int moe_abi_version(void);

/* The cudaError_t value behind the last MOE_ERR_CUDA returned on this host thread (0 if
 * none). */
int moe_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
