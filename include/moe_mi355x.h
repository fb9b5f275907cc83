/*
 * moe_mi355x.h -- C ABI of the routed mixture-of-experts expert-FFN hot path
 * and of the paged key-value cache and attention beside it, for AMD Instinct
 * MI355X (gfx950).
 *
 * Pages cited by title and section:
 *   [GATE-PR]  "Enable and fuse the Inkling MoE gate epilogue on Intel XPU"
 *              (sglang PR #36385)
 *   [CLAMP-PR] "[Moe] Fix flashinfer_trtllm silently dropping swiglu_limit
 *              clamped SwiGLU activation" (sglang PR #39920)
 *   [OAI-PR]   "fix(sm90): support parameterized SwiGLU in FP8 MegaMoE"
 *              (DeepGEMM PR #445)
 *   [INT4-PR]  "sm100: Fused INT4 grouped + SiLU Triton kernel"
 *              (batchgen PR #239)
 *   [LORA-AOT] "FlashInfer 0.6.18 SM100a+SM103a MoE-LoRA AOT -- SwiGLU LoRA
 *              up-delta units, EP scale lookups" (release notes); it serves
 *              NVFP4 expert weights with distinct gate/up global scales
 *
 * Conventions for every entry point:
 *   - Every array argument is DEVICE memory owned by the caller (plain
 *     pointers; the descriptors moe_weights / moe_lora / moe_layer /
 *     moe_act_params themselves are HOST structs read during the call).
 *     The library keeps no pointer after a call returns, allocates no device
 *     or host memory, and never synchronises except in
 *     moe_read_device_error. `stream` is a hipStream_t (NULL = default).
 *   - Work is enqueued asynchronously on `stream`; outputs are valid once the
 *     stream reaches that point.
 *   - Host-detectable problems return a negative moe_status and enqueue
 *     nothing. Launch failures return MOE_ERR_HIP (moe_last_error() has the
 *     HIP message). Data-dependent problems found on the device (a routing
 *     id outside [0, num_experts_global), a cache page that is not there) OR a MOE_DEVERR_* bit into a
 *     caller-owned int32 `err_word` (the caller zeroes it), skip the bad
 *     pair and leave every valid pair unaffected.
 *   - Row-major layouts; a "[G][N][K]" weight is G matrices of N output rows
 *     by K input columns.
 *   - Calls that share a workspace must not run concurrently.
 */
#ifndef MOE_MI355X_H
#define MOE_MI355X_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_NULL = -1,        /* a required pointer is NULL */
  MOE_ERR_SHAPE = -2,       /* a size is out of range or not a multiple */
  MOE_ERR_FORMAT = -3,      /* unknown weight format or format mismatch */
  MOE_ERR_LOCAL_RANGE = -4, /* missing/invalid local expert range */
  MOE_ERR_PARAM = -5,       /* non-finite or out-of-range scalar parameter */
  MOE_ERR_WORKSPACE = -6,   /* workspace NULL or too small */
  MOE_ERR_HIP = -8,         /* a HIP launch or runtime call failed */
  MOE_ERR_SCRATCH = -9      /* the call needs more than the static scratch of
                               moe_forward_no_workspace holds */
} moe_status;

typedef enum {
  MOE_W_BF16 = 0,      /* bf16 [G][N][K]; scale NULL */
  MOE_W_FP8_B128 = 1,  /* OCP e4m3fn [G][N][K]; scale fp32 [G][N/128][K/128]
                          (w = q * scale, 128x128 blocks) [CLAMP-PR
                          "Modifications": blockwise 128x128 FP8] */
  MOE_W_INT4_G32 = 2,  /* u8 [G][N][K/2] (byte j of a row: low nibble k=2j,
                          high nibble k=2j+1); scale bf16 [G][N][K/32];
                          w = (nibble - 8) * scale [INT4-PR commit text] */
  MOE_W_NVFP4 = 3,     /* e2m1 codes packed like INT4, u8 [G][N][K/2];
                          scale e4m3fn u8 [G][N][K/16]; w = e2m1(code) *
                          e4m3(scale) * gscale [LORA-AOT "Changes since
                          1b699bf": per-half NVFP4 global scales]. e2m1:
                          sign bit 3, magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6.
                          NaN scale codes (0x7F, 0xFF) set
                          MOE_DEVERR_W4_SCALE. */
  MOE_W_MXFP4 = 4,     /* e2m1 codes as NVFP4; scale e8m0 u8 [G][N][K/32];
                          w = e2m1(code) * 2^(scale - 127). Exact for scale
                          exponents 104..128 (2^-23 .. 2); a call that meets
                          another exponent sets MOE_DEVERR_W4_SCALE (its
                          outputs are then not valid). */
  MOE_W_MXFP4_A8 = 5   /* W4A8: the weights exactly as MOE_W_MXFP4, but the
                          activations enter GEMM1 as MXFP8 (see
                          moe_quantize_act_mxfp8) and GEMM1 runs on the
                          block-scaled matrix instructions, which take the
                          whole e8m0 range (code 0xFF, NaN, sets
                          MOE_DEVERR_W4_SCALE). Its 128-deep sums are
                          accurate to about 2e-5 of their sum of |products|
                          (not fp32-accurate); h is bf16 and GEMM2 is the
                          MOE_W_MXFP4 one. A choice of this library: the
                          pages fix no activation format for 4-bit weights. */
} moe_wfmt;

/* err_word bits */
#define MOE_DEVERR_GLOBAL_ID_OOB 0x1 /* a routing id < 0 or >= num_experts_global */
#define MOE_DEVERR_F16_RANGE 0x2     /* 4-bit layer: a bf16 activation x or h with
                                        |v| > 65504 (or not finite), beyond the f16
                                        operands of its matrix cores; the outputs
                                        of that call are not valid */
#define MOE_DEVERR_W4_SCALE 0x4      /* 4-bit layer: a weight scale outside the
                                        range the kernels expand exactly: INT4 a
                                        nonzero |scale| outside [2^-13, 2^13),
                                        NVFP4 a NaN e4m3 code, MXFP4 an exponent
                                        outside 104..128; outputs not valid */

/* Parameterized SwiGLU [CLAMP-PR "Modifications"; OAI-PR "Summary",
 * "Compatibility"]:
 *   g' = min(g, limit), u' = clamp(u, -limit, limit),
 *   h  = g' * sigmoid(alpha * g') * (u' + beta).
 * Defaults alpha = 1, beta = 0, limit = +INFINITY (no clamp) give
 * silu(g) * u. alpha and beta must be finite, limit > 0 (may be +inf). */
typedef struct {
  float alpha, beta, limit;
} moe_act_params;

/* One stacked expert weight (W13 = fused [gate | up], or W2 = down). */
typedef struct {
  int fmt;              /* moe_wfmt */
  int n_groups;         /* G: stacked matrices (local experts [+ shared]) */
  int N, K;             /* each matrix is [N][K]: W13 N = 2I, K = H;
                           W2 N = H, K = I */
  const void *q;        /* codes, layout per moe_wfmt */
  const void *scale;    /* scales, layout per moe_wfmt (NULL for BF16) */
  const float *gscale;  /* nullable. W13: fp32 [G][2] = (gate, up)
                           per-expert global scales multiplying the dequantised
                           gate rows 0..I-1 and up rows I..2I-1; the "true
                           units" of [LORA-AOT "Changes since 1b699bf"].
                           W2: NVFP4 / MXFP4 only (else MOE_ERR_FORMAT),
                           fp32 [G], one per expert. */
} moe_weights;
/* Alignment (MOE_ERR_PARAM): 4-bit codes 16 bytes; INT4 and NVFP4 scales
 * 2 bytes. Activations of 4-bit layers enter the matrix cores as f16:
 * exact for |x| in [2^-14, 65504] (and h alike); larger magnitudes set
 * MOE_DEVERR_F16_RANGE, smaller ones lose low bits (an absolute error below
 * 2^-25 per element). */

/* Rank-r LoRA of the local experts [LORA-AOT "Changes since 1b699bf"].
 * On the fused gate/up projection ("lora"): z = x A_e^T (fp32),
 * delta = scale * z B_e^T, added to g and u after each half's own global
 * scale, before the clamp.  A: bf16 [n_groups][rank][H], B: bf16
 * [n_groups][2I][rank].
 * On the down projection ("lora_down"): its input is activation_lora_input,
 * the SwiGLU output h in those true units rounded to bf16 (before any FP8
 * re-quantisation); z2 = h A2_e^T (fp32), y += scale * z2 B2_e^T, added to
 * the expert's output row before the routing-weighted combine.  A2: bf16
 * [n_groups][rank][I], B2: bf16 [n_groups][H][rank].
 * The shared expert (group E_loc) carries no LoRA.
 * A batch of adapters (n_adapters > 1; the page's harness serves eight
 * rank-16 adapters at once): A and B gain a leading adapter dimension,
 * [n_adapters][n_groups][...], and adapter_ids (device int32 [T], per call)
 * gives each token's adapter; a token whose id is outside [0, n_adapters)
 * gets no delta. n_adapters 0 or 1: one adapter for every token,
 * adapter_ids unused. A and B must be 16-byte aligned (MOE_ERR_PARAM). */
typedef struct {
  int rank;             /* 1..32 */
  int n_groups;         /* adapters for groups 0..n_groups-1 (the local
                           routed experts); later groups have none */
  float scale;
  const void *A;
  const void *B;
  int n_adapters;       /* 0..1024 */
  const int *adapter_ids;
} moe_lora;

/* ---------------------------------------------------------------- route -- */
/* Sigmoid-gate top-k with log-sigmoid renormalisation and shared-sink
 * columns [GATE-PR "2. Correctness", "3. Performance", router-epilogue
 * commit message]. Per token row t of `logits` (fp32, row stride `ld`
 * elements, ld >= n_routed + n_sink):
 *   - top_k passes of masked argmax over the n_routed leading columns,
 *     ranked on the raw logit when sel_bias is NULL (sigmoid is monotone),
 *     else on the fp32 key sigmoid(x) + sel_bias[c] (sel_bias fp32
 *     [n_routed]; the sink columns take no bias and never rank); equal keys
 *     resolve to the lower column index;
 *   - the winners carry their RAW logits: lp = logsigmoid of the k winners'
 *     raw logits and of the n_sink trailing sink columns; w = exp(lp -
 *     logsumexp(lp)) * route_scale * global_scale (finite when every logit
 *     is far below -104).
 * Outputs: topk_ids int32 [T][top_k] (global column ids, selection order),
 * topk_w fp32 [T][top_k], sink_w fp32 [T][n_sink] (NULL iff n_sink == 0),
 * packed int32 [T][top_k] or NULL: (id << 16) | bf16 bits of topk_w
 * (round to nearest even); a consumer takes the id as p >> 16 and the
 * weight from p & 0xFFFF.
 * Limits: 1 <= top_k <= n_routed, top_k + n_sink <= 64,
 * n_routed + n_sink <= 1024, T >= 0. Logits are assumed finite. */
int moe_route(const float *logits, long T, long ld, int n_routed, int n_sink,
              int top_k, const float *sel_bias, float route_scale,
              float global_scale, int *topk_ids, float *topk_w, float *sink_w,
              int *packed, void *stream);

/* ----------------------------------------------------------- gate route -- */
/* The router GEMM fused with the epilogue of moe_route [GATE-PR: the
 * "258-column gate GEMM" whose fp32 [T, N + S] rows feed the epilogue;
 * router-epilogue commit message]. logits[t][c] = sum_h x[t][h] * wg[c][h]
 * for c < n_routed + n_sink, bf16 operands, fp32 accumulation (in an order
 * of the kernel's choosing), then exactly the moe_route epilogue on those
 * rows (selection bias, raw-logit carry, sinks, scales, packed output).
 *   x_bf16   bf16 [T][H], row-major, 16-byte aligned;
 *   wg_bf16  bf16 [n_routed + n_sink][H] (routed rows first, then the sink
 *            rows), 16-byte aligned;
 *   logits   fp32 [T][n_routed + n_sink] or NULL (the gate rows, if the
 *            caller wants them);
 *   topk_ids, topk_w, sink_w, packed, sel_bias as for moe_route;
 *   ws       device workspace of moe_gate_route_workspace_size(T, H,
 *            n_routed, n_sink) bytes (0 when T is large enough for the
 *            single fused launch; NULL allowed then).
 * Limits: H a multiple of 32, 1 <= top_k <= n_routed, top_k + n_sink <= 16,
 * n_routed + n_sink <= 512, T >= 0 (T = 0 is a no-op). Errors: SHAPE for
 * the limits, NULL for a missing required pointer, PARAM for non-finite
 * scales or misaligned x / wg, WORKSPACE for a missing or short ws. */
size_t moe_gate_route_workspace_size(long T, int H, int n_routed, int n_sink);
int moe_gate_route(const void *x_bf16, const void *wg_bf16, long T, int H,
                   int n_routed, int n_sink, int top_k, const float *sel_bias,
                   float route_scale, float global_scale, float *logits,
                   int *topk_ids, float *topk_w, float *sink_w, int *packed,
                   void *ws, size_t ws_bytes, void *stream);

/* -------------------------------------------------------------- permute -- */
/* Expert-parallel rebase and grouping of (token, slot) pairs by local expert
 * [LORA-AOT "Changes since 1b699bf": ids are global, per-expert tables are
 * rank-local, rebase by local_expert_offset and bounds-check against the
 * local count; INT4-PR: per-expert sorted-token dispatch].
 *   pair id p = t*top_k + j; e = topk_ids[p] - local_expert_offset; the pair
 *   is local iff 0 <= e < num_local_experts. With shared_expert = 1 an
 *   always-on group G-1 = num_local_experts holds pairs p = T*top_k + t.
 *   Groups are laid out in order, pairs inside a group by ascending p.
 * Outputs: offsets int32 [G+1] (group g owns sorted rows
 * offsets[g]..offsets[g+1]-1), sorted_pair int32 [P_cap] (pair id of each
 * sorted row), pair_row int32 [T*top_k + shared*T] (sorted row of each pair
 * or -1), with P_cap = T*top_k + shared*T and G = num_local_experts +
 * shared_expert. Ids outside [0, num_experts_global) set
 * MOE_DEVERR_GLOBAL_ID_OOB in *err_word and are skipped.
 * Errors: MOE_ERR_LOCAL_RANGE unless num_local_experts >= 1,
 * local_expert_offset >= 0 and offset + num_local_experts <=
 * num_experts_global; MOE_ERR_SHAPE if G > 1024 or T*top_k >= 2^30.
 * Workspace: moe_permute_workspace_size(T, top_k, G) bytes. */
int moe_permute(const int *topk_ids, long T, int top_k, int num_experts_global,
                int local_expert_offset, int num_local_experts,
                int shared_expert, int *offsets, int *sorted_pair,
                int *pair_row, int *err_word, void *ws, size_t ws_bytes,
                void *stream);
size_t moe_permute_workspace_size(long T, int top_k, int n_groups);

/* -------------------------------------------------- activation quantise -- */
/* Per token and per 128-column group: amax in fp32, s = amax / 448 (s = 1
 * when amax == 0), q = e4m3fn(round-to-nearest-even(x / s)) saturated to
 * +-448 [CLAMP-PR "Modifications": the activation side of blockwise FP8].
 * x bf16 [T][H] -> xq e4m3fn [T][H], xs fp32 [T][H/128]. H % 128 == 0. */
int moe_quantize_act_fp8(const void *x_bf16, long T, int H, void *xq,
                         float *xs, void *stream);

/* MXFP8 activations, the GEMM1 input of MOE_W_MXFP4_A8 layers: per token and
 * per 32 columns, amax in fp32, e = the smallest integer with
 * amax <= 448 * 2^e (raised to -127 when smaller, e.g. an all-zero group),
 * xe = e + 127 (e8m0), xq = e4m3fn(round-to-nearest-even(x / 2^e)) (never
 * beyond 448, so never saturated). x bf16 [T][H] -> xq e4m3fn [T][H] +
 * xe u8 [T][H/32]. H % 128 == 0. */
int moe_quantize_act_mxfp8(const void *x_bf16, long T, int H, void *xq,
                           void *xe, void *stream);

/* ------------------------------------------------ grouped GEMM1 + SwiGLU -- */
/* err_word of the GEMM entry points: device int32, ORed with the
 * MOE_DEVERR_F16_RANGE / MOE_DEVERR_W4_SCALE bits a 4-bit layer meets
 * (required for 4-bit weights: MOE_ERR_NULL without it; nullable, and
 * never written, for BF16 and FP8 weights). */
/* For each group g and each of its sorted rows r (token t of pair
 * sorted_pair[r]):  [g | u] = x_t W13_g^T  (fp32 accumulation;
 * FP8: per 128-K block partial sums times xs[t][kb] * scale[g][nb][kb]),
 * times gscale[g] (gate, up) when given, plus the LoRA delta when given,
 * then the parameterized SwiGLU `act` -> h[r][0..I-1].
 *   FP8 weights: x = xq e4m3fn [T][H] with xs fp32 [T][H/128]; h is
 *     re-quantised like moe_quantize_act_fp8 per row and 128 columns:
 *     h e4m3fn [P_cap][I], hs fp32 [P_cap][I/128].
 *   MXFP4_A8 weights: x = xq e4m3fn [T][H] with xs = xe u8 [T][H/32]
 *     (moe_quantize_act_mxfp8); h bf16 as below, hs NULL.
 *   BF16 / other 4-bit (INT4, NVFP4, MXFP4) weights: x bf16 [T][H] (xs NULL);
 *     h bf16 [P_cap][I] (round-to-nearest-even), hs NULL.
 * x_bf16 bf16 [T][H] is the LoRA input (NULL without LoRA).
 * h_lora (FP8 weights only, else it must be NULL: MOE_ERR_PARAM), nullable:
 * bf16 [P_cap][I], the SwiGLU output before the re-quantisation (round to
 * nearest even), i.e. the down-LoRA input; BF16 / 4-bit layers pass h itself
 * to moe_grouped_gemm2_combine instead.
 * offsets / sorted_pair come from moe_permute for the same (T, top_k);
 * w13->n_groups = G, w13->N = 2I, w13->K = H. p_cap = rows allocated in h.
 * Limits: H % 128 == 0 and I % 128 == 0. Workspace:
 * moe_gemm1_workspace_size(w13, p_cap, lora) bytes: the LoRA z rows; for
 * FP8 / 4-bit weights at decode sizes (few enough tiles of 32 rows x 128 h
 * columns that one tile per workgroup would leave CUs idle) the fp32
 * partial sums of a split-K schedule (4 * p_cap * 2I floats), which spreads
 * the K blocks of those tiles over all CUs and reduces them in a fixed
 * order; for 4-bit weights other than MXFP4_A8 the f16 copy of the
 * activations (p_cap * H * 2 bytes, T <= p_cap). Returns 0 for a NULL w13 or N not a multiple of 256. */
int moe_grouped_gemm1_act(const moe_weights *w13, const void *x,
                          const void *xs, const void *x_bf16, long T, int H,
                          int I, int top_k, long p_cap, const int *offsets,
                          const int *sorted_pair, const moe_act_params *act,
                          const moe_lora *lora, void *h, float *hs,
                          void *h_lora, int *err_word, void *ws,
                          size_t ws_bytes, void *stream);
size_t moe_gemm1_workspace_size(const moe_weights *w13, long p_cap,
                                const moe_lora *lora);

/* ---------------------------------------- grouped GEMM2 + weighted combine -- */
/* y[r] = h[r] W2_g^T (fp32; FP8 per 128-K block partial sums times
 * hs[r][kb] * scale[g][nb][kb]; FP4 times w2->gscale[g] when given) for
 * every sorted row, plus with lora_down
 * the down-LoRA delta scale * (h_lora[r] A2_g^T) B2_g^T for groups
 * g < lora_down->n_groups (h_lora bf16 [P_cap][I]: GEMM1's h_lora output
 * for FP8 weights, h itself for BF16 / 4-bit weights). For FP8 and 4-bit
 * weights the rows y pass to the combine in block floating point: one
 * power-of-two scale per row and 16 columns and an int16 multiple of it per
 * value, rounded to nearest (error at most 2^-15 of the run's largest
 * magnitude; a value that is not finite becomes NaN); BF16 layers keep
 * fp32 rows. Then
 *   out[t][:] = sum_{j < top_k, pair_row[t*top_k+j] >= 0} topk_w[t][j] *
 *               y[pair_row[t*top_k+j]]   (ascending j, fp32)
 *             + shared_w * y[pair_row[T*top_k + t]]   (if shared_expert)
 * [INT4-PR: slot-specific routing-weight reduction, fp32 accumulation].
 * Every out element is written (0 for a token with no local pair).
 * w2->N = H, w2->K = I. out fp32 [T][H]. Limits: 1 <= top_k <= 64
 * (MOE_ERR_SHAPE). err_word as for moe_grouped_gemm1_act. Workspace:
 * moe_gemm2_workspace_size(w2, p_cap, lora_down) bytes: the y rows (and
 * their scale exponents), or
 * for FP8 / 4-bit weights at decode sizes their split-K partial sums
 * (4 * p_cap * H floats, reduced by the combine in a fixed order; the
 * down-LoRA delta enters the first partial of each tile), then the
 * down-LoRA z2 rows (p_cap * rank floats, plus p_cap ints with a batch of
 * adapters). sorted_pair (moe_permute's) is needed with lora_down only (it
 * maps rows to tokens for the adapter ids). Errors: NULL for a lora_down
 * without h_lora or sorted_pair. Returns 0 for a NULL w2. */
int moe_grouped_gemm2_combine(const moe_weights *w2, const void *h,
                              const float *hs, const void *h_lora,
                              const moe_lora *lora_down, long T, int H, int I,
                              int top_k, int shared_expert, long p_cap,
                              const int *offsets, const int *sorted_pair,
                              const int *pair_row, const float *topk_w,
                              float shared_w, float *out, int *err_word,
                              void *ws, size_t ws_bytes, void *stream);
size_t moe_gemm2_workspace_size(const moe_weights *w2, long p_cap,
                                const moe_lora *lora_down);

/* ---------------------------------------------------------- whole layer -- */
typedef struct {
  int H, I;
  int num_experts_global;   /* routed experts E (logit columns 0..E-1) */
  int num_local_experts;    /* experts held here, global ids
                               [offset, offset + num_local_experts) */
  int local_expert_offset;
  int shared_expert;        /* 0 | 1: always-on group num_local_experts */
  int top_k, n_sink;        /* n_sink trailing sink logit columns */
  float route_scale, global_scale, shared_w;
  moe_weights w13, w2;      /* n_groups = num_local_experts + shared_expert */
  moe_act_params act;
  const moe_lora *lora;     /* nullable: LoRA on [gate | up] */
  const moe_lora *lora_down;/* nullable: LoRA on the down projection, input
                               the true-units SwiGLU output (see moe_lora) */
} moe_layer;

/* One call of the whole path on `stream`: moe_route -> moe_permute ->
 * (FP8) moe_quantize_act_fp8 | (MXFP4_A8) moe_quantize_act_mxfp8 ->
 * moe_grouped_gemm1_act ->
 * moe_grouped_gemm2_combine. x_bf16 bf16 [T][H]; logits fp32 [T][ld_logits]
 * with ld_logits >= num_experts_global + n_sink. Outputs out fp32 [T][H],
 * topk_ids/topk_w [T][top_k], sink_w [T][n_sink] (NULL iff n_sink == 0),
 * err_word as in moe_permute and the GEMM entry points. Workspace: moe_workspace_size(layer, T_max)
 * bytes, T <= T_max. Errors: those of the steps, checked before any launch. */
int moe_forward(const moe_layer *layer, const void *x_bf16,
                const float *logits, long T, long ld_logits, float *out,
                int *topk_ids, float *topk_w, float *sink_w, int *err_word,
                void *ws, size_t ws_bytes, void *stream);
size_t moe_workspace_size(const moe_layer *layer, long T_max);

/* moe_forward for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same computation and the same kernels, with the workspace taken from
 * a static device array of MOE_SCRATCH_BYTES that the library holds on
 * every GPU it runs on, from module load until the process ends. Arguments
 * as for moe_forward without ws / ws_bytes; the caller still passes (and
 * owns) every input and output. The device is the current one; its
 * array's address is looked up on the first call there. A layer and T whose
 * moe_workspace_size exceeds MOE_SCRATCH_BYTES return MOE_ERR_SCRATCH
 * (moe_scratch_error() says how much was needed) and launch nothing; 32 MiB
 * holds every layer here at T <= 64. Calls on one GPU share its array:
 * calls that overlap on one GPU (two streams, two threads) race and must be
 * ordered by the caller. Nothing in the array has to start at zero (each
 * call writes every workspace byte before reading it). */
#define MOE_SCRATCH_BYTES (32u << 20)
int moe_forward_no_workspace(const moe_layer *layer, const void *x_bf16,
                             const float *logits, long T, long ld_logits,
                             float *out, int *topk_ids, float *topk_w,
                             float *sink_w, int *err_word, void *stream);
/* Message of the calling thread's last moe_forward_no_workspace refusal
 * ("" if none). */
const char *moe_scratch_error(void);

/* ------------------------------------------------------- key-value cache -- */
/* The other half of a decoder layer in serving: attention over a paged
 * key-value cache, the writing of new keys and values into it and the upkeep
 * of its pages. These follow from the formulas stated here (no page of the
 * sources above covers them).
 *
 * One layer's cache is two arrays of pages, K and V, of n_pages pages of
 * page_size tokens of n_heads key-value heads of head_dim values; value d of
 * head h of token i of page p lies at element
 *   p * stride_page + h * stride_head + i * stride_tok + d,
 * so both [page][head][token][d] and [page][token][head][d] are expressed.
 * Pages of several sequences are found through one moe_kv_table for all
 * layers: token j of slot s is token j % page_size of page
 * table[s * ld + j / page_size]; an entry outside [0, n_pages) (by
 * convention -1) holds no page. len[s] is the number of tokens of slot s,
 * the newest included. refs[p] counts the table entries that name page p;
 * pages with refs 0 are free. */
typedef enum {
  MOE_KV_BF16 = 0,
  MOE_KV_F16 = 1,
  MOE_KV_E4M3 = 2      /* OCP e4m3fn codes; value = code * scale[head] */
} moe_kv_fmt;

typedef struct {
  int fmt;             /* moe_kv_fmt */
  int n_pages;         /* >= 1 */
  int page_size;       /* a multiple of 16, 16..4096 */
  int n_heads;         /* key-value heads, 1..1024 */
  int head_dim;        /* 64, 128 or 256 */
  long stride_page, stride_head, stride_tok;   /* elements; multiples of 16
                          bytes, at least head_dim; stride_tok * 16 elements
                          under 2^30 bytes */
  void *k, *v;         /* 16-byte aligned */
  const float *k_scale, *v_scale;   /* device fp32 [n_heads]; MOE_KV_E4M3
                          only (NULL otherwise) */
} moe_kv_cache;

typedef struct {
  int n_slots;         /* rows of table, entries of len */
  int max_pages;       /* entries of a row; max_pages * page_size <= 2^28 */
  long ld;             /* row stride of table, >= max_pages */
  int n_pages;         /* as the cache's */
  int page_size;       /* as the cache's */
  int *table;          /* int32 [n_slots][ld] */
  int *len;            /* int32 [n_slots], 0..max_pages * page_size (what
                          lies outside is taken as the nearest bound) */
  int *refs;           /* int32 [n_pages]; NULL for attention and append,
                          which do not use it; never touched concurrently by
                          two calls */
} moe_kv_table;

/* err_word bits of the calls below (the word is required; moe_read_device_error
 * reads it) */
#define MOE_DEVERR_CACHE_PAGE 0x8  /* a token that a call reads or writes has no
                                      page, or a slot index is >= n_slots (that
                                      token is taken as masked, or not written;
                                      that slot as empty) */
#define MOE_DEVERR_CACHE_FULL 0x10 /* grow or fork: not enough free pages or
                                      table entries for a slot, left as it was */
#define MOE_DEVERR_CACHE_BUSY 0x20 /* fork into a slot that holds tokens, keep
                                      or grow in a page of several slots: left
                                      as it was */
#define MOE_DEVERR_TREE 0x40       /* a drafted token whose parent does not come
                                      before it (taken as a child of the
                                      context), a tree of more than
                                      MOE_TREE_MAX tokens (its rows give 0 and
                                      -infinity), or an accepted path that is
                                      none (that slot left as it was) */

/* Queries, outputs and mask of an attention call. Row r of q belongs to
 * position p of its sequence (see the entry points), query head h to
 * key-value head h / (n_heads / cache->n_heads). Key j is visible iff
 *   j <= p and (window == 0 or p - j < window or j < n_first):
 * causal, optionally within a sliding window of the last `window` keys, of
 * which the first n_first keys of the sequence stay visible. With
 * s_j = scale * sum_d q[d] K_j[d] over the visible keys,
 *   out = sum_j exp(s_j - lse) V_j,  lse = log sum_j exp(s_j);
 * a row that sees no key (or only scores of -infinity) gets out = 0 and
 * lse = -infinity. What lies in masked places, infinities and NaN included,
 * does not enter. Products accumulate in fp32, the softmax statistics are
 * fp32; the probabilities enter the second product in the type of q, all
 * those from 2^-26 of the largest on with its full precision (prompts in f16:
 * for scores up to 1.8e5). */
typedef struct {
  int fmt;             /* MOE_KV_BF16 or MOE_KV_F16: q and out; a cache that
                          is not MOE_KV_E4M3 has the same fmt */
  int n_heads;         /* a multiple of cache->n_heads, at most 64 times it */
  const void *q;       /* [rows][n_heads][head_dim], 16-byte aligned */
  long q_stride_row, q_stride_head;       /* elements, multiples of 8 */
  void *out;           /* as q */
  long out_stride_row, out_stride_head;
  float *lse;          /* fp32 [rows][n_heads], dense, or NULL */
  float scale;         /* finite */
  int window;          /* >= 0; 0: no window */
  int n_first;         /* >= 0; used with a window */
} moe_attn;

/* Attention of one new token per sequence: row i of q is the token at
 * position len[s] - 1 of slot s = slots[i] (slots NULL: s = i). A negative
 * slots[i] is a row without a sequence (out 0, lse -infinity), so a batch of
 * fixed size can be captured once and run partly filled. The visible keys of
 * all sequences and key-value heads are split evenly over the GPU, whatever
 * the lengths, and the parts of one sequence joined in a fixed order (a
 * second launch, left out where nothing can be split): results do not depend
 * on timing. No length is read on the host. Limits: 0 <= n < 2^20. Workspace:
 * moe_attn_decode_workspace_size(cache, n, n_heads) bytes (0 for invalid
 * arguments). Errors: NULL, SHAPE, FORMAT (fmt), PARAM (alignment, scale,
 * window, scales of a cache that takes none), WORKSPACE, HIP. */
int moe_attn_decode(const moe_kv_cache *cache, const moe_kv_table *table,
                    const int *slots, long n, const moe_attn *attn,
                    int *err_word, void *ws, size_t ws_bytes, void *stream);
size_t moe_attn_decode_workspace_size(const moe_kv_cache *cache, long n,
                                      int n_heads);

/* Attention of the newest tokens of n sequences: rows cu_q[i] ..
 * cu_q[i + 1] - 1 of q (device int32 [n + 1], ascending from 0 to T) are the
 * last m = cu_q[i + 1] - cu_q[i] tokens of slot s = slots[i] (NULL: s = i),
 * row cu_q[i] + t at position len[s] - m + t; rows outside cu_q[0] ..
 * cu_q[n] - 1 are not written. A whole prompt (m = len) or the
 * next chunk of one; its keys and values are in the cache already
 * (moe_cache_append). Rows with a negative slots[i] or position give 0 and
 * -infinity. T = rows of q (< 2^31 / n_heads). Workspace:
 * moe_attn_prefill_workspace_size(cache, n, T, n_heads) bytes. Errors
 * as for moe_attn_decode. */
int moe_attn_prefill(const moe_kv_cache *cache, const moe_kv_table *table,
                     const int *slots, long n, const int *cu_q, long T,
                     const moe_attn *attn, int *err_word, void *ws,
                     size_t ws_bytes, void *stream);
size_t moe_attn_prefill_workspace_size(const moe_kv_cache *cache, long n,
                                       long T, int n_heads);

/* Attention of drafted tokens that form a tree behind the context of each
 * sequence. As moe_attn_prefill: rows cu_q[i] .. cu_q[i + 1] - 1 of q are the
 * last m tokens of slot s = slots[i], at most MOE_TREE_MAX of them, their keys
 * and values in the cache already. parent[r] (device int32 [T]) is row r's
 * parent as an index among its sequence's rows, before its own (0 .. t - 1 for
 * the t-th row), or -1: a child of the context. Row t sees, of the C = len[s] -
 * m tokens before, all, and of the drafted ones itself and its ancestors. The
 * position of a drafted token is C + the number of its ancestors: with a
 * window the key at position p is visible to the row at position p' iff
 * p' - p < window or p < n_first. A sequence with len[s] < m gives 0 and
 * -infinity. After the verdict over the tree: moe_cache_keep. Workspace:
 * moe_attn_tree_workspace_size(cache, n, T, n_heads) bytes. Errors as for
 * moe_attn_decode. */
#define MOE_TREE_MAX 256
int moe_attn_tree(const moe_kv_cache *cache, const moe_kv_table *table,
                  const int *slots, long n, const int *cu_q, long T,
                  const int *parent, const moe_attn *attn, int *err_word,
                  void *ws, size_t ws_bytes, void *stream);
size_t moe_attn_tree_workspace_size(const moe_kv_cache *cache, long n, long T,
                                    int n_heads);

/* Writes new keys and values: rows cu[i] .. cu[i + 1] - 1 of k and v (device
 * int32 [n + 1]; NULL: one row each, T = n) go to positions start[i],
 * start[i] + 1, ... of slot slots[i] (NULL: i). Nothing is written for a
 * negative start[i] or slots[i]. k and v: [T][n_heads][head_dim] of type fmt
 * (MOE_KV_BF16 or MOE_KV_F16; the cache's own unless that is MOE_KV_E4M3),
 * 16-byte aligned, strides in elements, multiples of 8. Into a MOE_KV_E4M3
 * cache: code = e4m3fn(round-to-nearest-even(x / scale[head])), the fp32
 * quotient saturated to +-448 (NaN: 0x7F). Positions of different rows must
 * differ, and lie in pages that no other slot's table names, as those that
 * moe_cache_grow gives do. */
int moe_cache_append(const moe_kv_cache *cache, const moe_kv_table *table,
                     const int *slots, const int *start, const int *cu, long n,
                     long T, int fmt, const void *k, long k_stride_row,
                     long k_stride_head, const void *v, long v_stride_row,
                     long v_stride_head, int *err_word, void *stream);

/* Upkeep of the pages. The slots of one call are distinct and valid. One
 * call's table is not used by another stream meanwhile. Pages are taken
 * lowest index first, in the order of the list: results do not depend on
 * timing.
 *
 * moe_cache_grow makes room for n_new[i] >= 0 more tokens of slots[i] (NULL:
 * i) and counts them in: start[i] = len, len += n_new[i], with new pages
 * where page_size * (entries held) is short. A slot is left as it was, with
 * start[i] = -1 and MOE_DEVERR_CACHE_FULL, if its table row is too short, or
 * if it needs a page and the slots up to it in the list whose rows suffice
 * need more pages in all than are free; with MOE_DEVERR_CACHE_BUSY if it is to
 * get tokens (n_new[i] > 0) and ends inside a page that other entries name too
 * (refs > 1; moe_cache_keep may cut a slot back to there), where they would be
 * written over theirs. It needs no pages in that count then. A fork of it goes on in a copy of that
 * page, and so does the slot itself once no other has the page.
 *
 * moe_cache_free gives the slots' pages back (refs - 1 each, entries -1,
 * len 0), those in entries past the tokens too. (Grow and fork expect none
 * there: grow writes over such entries, fork leaves them out.)
 * moe_cache_trim gives back the pages whose tokens j all have
 * n_first <= j < len - window (no query from position len - 1 on sees them),
 * entries -1, len unchanged.
 *
 * moe_cache_fork makes dst[i], an empty slot, a copy of src[i]: whole pages
 * are shared (refs + 1), a partly filled last page is copied into a free
 * page, in every layer, since both go on writing there. dst entries are
 * distinct and none of them a src. If no page is free, dst[i] stays empty,
 * with MOE_DEVERR_CACHE_FULL.
 *
 * moe_cache_compact moves pages, in every layer, so that the pages in use
 * are the first ones: with U pages in use, the i-th of those at index >= U
 * moves to the i-th free page below U; refs and every table entry follow.
 * n_used[0] = U (device int32, NULL allowed).
 *
 * moe_cache_keep keeps the accepted path of each tree of drafted tokens
 * (moe_attn_tree): of the n_draft[i] newest tokens of slots[i] (NULL: i), those
 * at path[cu[i]] .. path[cu[i + 1] - 1] among them (device int32 [n_path];
 * ascending, as a path from the context down is) become the next ones behind
 * the context, in every layer; the slot's length follows, and pages left
 * without tokens go back. An entry that is no such path leaves its slot as it
 * was, with MOE_DEVERR_TREE; so does one that would write into a page of
 * another slot too, with MOE_DEVERR_CACHE_BUSY. A path that moves nothing
 * writes nothing, and may leave the slot's end inside such a page (see
 * moe_cache_grow). cu: device int32 [n + 1], within 0..n_path.
 *
 * moe_cache_copy_pages copies page src[i] to page dst[i], in every layer;
 * entries < 0 are skipped, entries >= n_pages too, with
 * MOE_DEVERR_CACHE_PAGE. No dst occurs twice or is also a src.
 *
 * layers: host array of n_layers (1..1024) caches alike in all but their
 * pointers and scales; a cache whose v is its k has one array. Limits: 0 <= n <
 * 2^20, for fork 0 <= n <= 65535, for copy_pages 0 <= n < 2^31, for keep 0 <=
 * n_path < 2^31. Workspace: moe_cache_workspace_size(table, n) bytes, 16-byte
 * aligned, serve grow, fork and compact for up to n slots; keep takes none. */
int moe_cache_grow(const moe_kv_table *table, const int *slots,
                   const int *n_new, long n, int *start, int *err_word,
                   void *ws, size_t ws_bytes, void *stream);
int moe_cache_free(const moe_kv_table *table, const int *slots, long n,
                   int *err_word, void *stream);
int moe_cache_trim(const moe_kv_table *table, const int *slots, long n,
                   int window, int n_first, int *err_word, void *stream);
int moe_cache_fork(const moe_kv_cache *layers, int n_layers,
                   const moe_kv_table *table, const int *src, const int *dst,
                   long n, int *err_word, void *ws, size_t ws_bytes,
                   void *stream);
int moe_cache_compact(const moe_kv_cache *layers, int n_layers,
                      const moe_kv_table *table, int *n_used, int *err_word,
                      void *ws, size_t ws_bytes, void *stream);
int moe_cache_keep(const moe_kv_cache *layers, int n_layers,
                   const moe_kv_table *table, const int *slots,
                   const int *n_draft, const int *cu, const int *path,
                   long n_path, long n, int *err_word, void *stream);
int moe_cache_copy_pages(const moe_kv_cache *layers, int n_layers,
                         const int *src, const int *dst, long n, int *err_word,
                         void *stream);
size_t moe_cache_workspace_size(const moe_kv_table *table, long n);

/* ------------------------------------------------------- latent attention -- */
/* Attention whose keys and values are one latent vector a token, shared by all
 * query heads: with c_j the latent vector of token j (latent_dim values) and
 * r_j its rotary key (rope_dim values), head h's key is [Wk_h c_j, r_j] and its
 * value Wv_h c_j. A cache keeps c_j and r_j alone, in one array of pages: value
 * d of token i of page p lies at element p * stride_page + i * stride_tok + d,
 * the rotary values behind the latent ones. Its tables are moe_kv_table; grow,
 * free and trim take them as they are, fork, compact, keep and copy_pages
 * take the array as moe_latent_pages describes it. */
typedef struct {
  int fmt;             /* moe_kv_fmt */
  int n_pages;         /* >= 1 */
  int page_size;       /* a multiple of 16, 16..4096 */
  int latent_dim;      /* 256 or 512 */
  int rope_dim;        /* 64 */
  long stride_page, stride_tok;   /* elements; multiples of 16 bytes, at least
                          latent_dim + rope_dim; stride_tok * 16 elements under
                          2^30 bytes */
  void *c;             /* 16-byte aligned */
  const float *scale;  /* device fp32 [1], value = code * scale; MOE_KV_E4M3
                          only (NULL otherwise) */
} moe_latent_cache;

/* The cache as the calls that move pages take it: heads of 64 values and no
 * second array (v = k). Not for attention or append. */
int moe_latent_pages(const moe_latent_cache *cache, moe_kv_cache *pages);

/* Writes new tokens, as moe_cache_append: rows of c [T][latent_dim] and of rope
 * [T][rope_dim], of type fmt, strides of their rows in elements, multiples of
 * 8. */
int moe_latent_append(const moe_latent_cache *cache, const moe_kv_table *table,
                      const int *slots, const int *start, const int *cu, long n,
                      long T, int fmt, const void *c, long c_stride_row,
                      const void *rope, long rope_stride_row, int *err_word,
                      void *stream);

/* Absorbed attention over the cache: with q'_h = [Wk_h^T q_h, q_rope_h] the
 * scores are those of the keys [c_j, r_j], and the result is sum_j p_j c_j, from
 * which the caller takes Wv_h times it. attn: q [rows][n_heads][latent_dim +
 * rope_dim], out [rows][n_heads][latent_dim], n_heads 1..1024, the rest as for
 * moe_attn_prefill. Rows cu_q[i] .. cu_q[i + 1] - 1 (device int32 [n + 1]; NULL:
 * one row each, T = n) are the newest tokens of slots[i] (NULL: i): what they
 * see of each other goes by parent as in moe_attn_tree, or, without (NULL), by
 * their order as in moe_attn_prefill. The keys of all rows are dealt out evenly
 * over the GPU and the parts joined in a fixed order. A key that is not finite
 * makes the rows that see it NaN, unless it gives them a score of -infinity and
 * with it no part in the sum. Limits: 0 <= n < 2^20,
 * T < 2^31 / n_heads. Workspace: moe_attn_latent_workspace_size(cache, n, T,
 * n_heads) bytes (34 MB for vectors of 256 and 68 for 512, whatever the batch).
 * Errors as for moe_attn_decode. */
int moe_attn_latent(const moe_latent_cache *cache, const moe_kv_table *table,
                    const int *slots, long n, const int *cu_q, long T,
                    const int *parent, const moe_attn *attn, int *err_word,
                    void *ws, size_t ws_bytes, void *stream);
size_t moe_attn_latent_workspace_size(const moe_latent_cache *cache, long n,
                                      long T, int n_heads);

/* Expanded attention of prompts: head h's keys are [k[j][h], k_rope[j]] and its
 * values v[j][h], as a product of Wk_h and Wv_h with the latent vectors left
 * them, in rows instead of pages. */
typedef struct {
  const void *k;       /* [S][n_heads][128], 16-byte aligned */
  long k_stride_row, k_stride_head;    /* elements, multiples of 8; strides of
                          rows under 2^25 */
  const void *k_rope;  /* [S][64], shared by the heads */
  long rope_stride_row;
  const void *v;       /* [S][n_heads][128] */
  long v_stride_row, v_stride_head;
} moe_latent_rows;

/* attn: q [T][n_heads][192] (128 values for k, then 64 for k_rope), out
 * [T][n_heads][128], n_heads 1..1024, window and n_first as for
 * moe_attn_prefill; rows all of type fmt. Rows cu_q[i] .. cu_q[i + 1] - 1 of q
 * are the newest tokens of the sequence whose keys and values are rows cu_k[i]
 * .. cu_k[i + 1] - 1 (device int32 [n + 1] each, ascending, cu_k from 0 to S <=
 * 2^28): a prompt, or, with more keys than rows, the next chunk of one. Rows of
 * q before their sequence's first key give 0 and -infinity; rows outside the
 * list are not written. Workspace: moe_attn_latent_prompt_workspace_size(n, T,
 * n_heads) bytes. Errors: NULL, SHAPE, FORMAT, PARAM, WORKSPACE, HIP. */
int moe_attn_latent_prompt(const moe_latent_rows *kv, long n, const int *cu_k,
                           long S, const int *cu_q, long T,
                           const moe_attn *attn, void *ws, size_t ws_bytes,
                           void *stream);
size_t moe_attn_latent_prompt_workspace_size(long n, long T, int n_heads);

/* --------------------------------------------------------------- misc -- */
/* Synchronises `stream`, then copies *err_word (device) to *host_bits. */
int moe_read_device_error(const int *err_word, int *host_bits, void *stream);
const char *moe_status_string(int status);
/* Last HIP error message of the calling thread ("" if none). */
const char *moe_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_H */
