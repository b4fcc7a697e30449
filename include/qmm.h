/*
 * qmm.h - C ABI of the MI355X (gfx950) weight-quantized GEMV / GEMM library.
 *
 * What the library computes
 * -------------------------
 * BaseRT (native-Metal LLM inference on Apple Silicon), §3.3 "kernel fusion
 * and specialization": matrix multiplies over group-quantized weights, one
 * GEMV variant for decode (M = 1) and one GEMM variant for prefill (M > 1),
 * with dequantization folded into the inner loop so that dequantized
 * weights never reach memory.  §3.4 "prefill": the M > 1 case is a tiled
 * GEMM on [seq_len x dim] activations and is compute-bound.  The abstract
 * and Fig. 1 add mixture-of-experts prefill (Qwen3-30B-A3B), served here by
 * a grouped GEMM over token-to-expert buckets.  §3 states that the runtime
 * is reached through a C API, and §3.2 that the decode loop allocates
 * nothing and reports errors through static thread-local buffers; this ABI
 * follows both.
 *
 * For every entry point, with W_hat[n, k] = s[n, k/gs] * q[n, k] + b[n, k/gs]:
 *     y[m, n] = sum_k x[m, k] * W_hat[n, k]          (fp32 accumulation)
 *
 * Data formats (all little-endian, all row-major)
 * ----------------------------------------------
 *   weights  W[n, k] is [out, in].  Codes q in 0 .. 2^bits - 1 are packed
 *            along k as a little-endian bit stream: code k occupies bits
 *            [bits*k, bits*k + bits) of its row, bit i of the stream is bit
 *            i % 32 of uint32 word i / 32.  For bits = 4 that is 8 nibbles per
 *            word, low nibble first; for bits = 8, 4 bytes per word, low byte
 *            first; 3-, 5- and 6-bit codes straddle word boundaries (every 8
 *            codes fill exactly `bits` bytes).  Row stride: k * bits / 32
 *            words; a 64-code group is 8 * bits bytes.  The GEMM entry points
 *            also read a tile-interleaved copy of these words (see
 *            qmm_repack_tiled and QMM_WEIGHTS_TILED).
 *   scales,  fp16 bit patterns (uint16) [n, k / group_size]: the per-group
 *   biases   step s and offset b (asymmetric min/max quantization: b is the
 *            group minimum, s = (max - min) / (2^bits - 1)).
 *   x        fp16 bit patterns, [m, k].
 *   y        fp32, [m, n].
 *
 * Common rules
 * ------------
 *   * Supported: bits in {2, 3, 4, 5, 6, 8}; group_size in {32, 64, 128}; k a positive
 *     multiple of 64 and of group_size; n, m >= 1 (m = 0 / t = 0 is accepted and does nothing).
 *   * Every tensor pointer is a DEVICE pointer owned by the caller and must
 *     stay valid until the stream reaches the launch.  Weights, activations,
 *     plans and workspaces must be 16-byte aligned; scales and biases 2-byte
 *     aligned (8-byte aligned arrays let the GEMM kernels load the scales of
 *     four groups at once; others take a slower per-group path); outputs
 *     4-byte (fp32) or 2-byte (fp16) aligned.
 *     Output buffers must not overlap inputs.
 *   * `stream` is a hipStream_t (NULL = the null stream).  Calls enqueue
 *     work and return; results are valid once the stream is synchronized.
 *   * No entry point allocates device memory, frees it or synchronizes.
 *     Scratch memory comes from a caller-provided workspace whose size the
 *     matching *_workspace_size query returns.
 *   * Arguments are validated on the host before any HIP call, so every
 *     error status below can be produced without a GPU.  On error nothing is
 *     launched and qmm_last_error() describes the problem.
 *   * Thread safety: stateless apart from a thread-local error message;
 *     calls from several threads on several streams are safe.
 */
#ifndef QMM_H
#define QMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QMM_OK = 0,
  QMM_ERR_INVALID_ARG = 1,  /* null / misaligned pointer, bad size, k % group_size != 0 */
  QMM_ERR_UNSUPPORTED = 2,  /* bits or group_size outside the supported set */
  QMM_ERR_WORKSPACE = 3,    /* workspace or plan buffer too small */
  QMM_ERR_HIP = 4           /* a HIP launch failed; text in qmm_last_error() */
} qmm_status;

/* hipStream_t, passed as an opaque pointer so that this header needs no HIP headers. */
typedef void* qmm_stream;

/* Library version, major * 10000 + minor * 100 + patch. */
int qmm_version(void);

/* Text of the last error raised on the calling thread ("" if none).  The
 * buffer is thread-local and static (BaseRT §3.2); it stays valid until the
 * next qmm_* call on the same thread. */
const char* qmm_last_error(void);

/* ------------------------------------------------------------ decode GEMV
 * y[n] = sum_k x[k] * W_hat[n, k]   (BaseRT §3.3: the M = 1 decode kernel)
 *   w       [n, k*bits/32] uint32 packed codes
 *   scales  [n, k/group_size] fp16 bits;  biases likewise
 *   x       [k] fp16 bits;  y [n] fp32 (overwritten)
 * Streams every weight byte once with 128-bit loads, unpacks and scales in
 * registers, reduces across lanes; small n gets an in-workgroup split of k.
 * Errors: INVALID_ARG, UNSUPPORTED, HIP. */
int qmm_qgemv(const uint32_t* w, const uint16_t* scales, const uint16_t* biases,
              const uint16_t* x, float* y, int n, int k, int bits, int group_size,
              qmm_stream stream);

/* ---------------------------------------------------- batched decode GEMV
 * Many independent GEMVs (e.g. every projection of a decode step) in ONE
 * launch, which amortizes launch cost the way BaseRT §3 amortizes command
 * dispatch.  Two steps:
 *   1. qmm_qgemv_batched_plan (host only, no HIP call): from `count` problem
 *      descriptors (device pointers inside, host array) build a plan image
 *      in host memory `plan` of `plan_bytes`.  *plan_bytes_needed receives
 *      the size required; if plan is NULL or too small the call returns
 *      QMM_ERR_WORKSPACE without writing the plan.  All problems share bits
 *      and group_size; each has its own n and k.
 *   2. Copy the image verbatim to device memory (any copy), then call
 *      qmm_qgemv_batched with the device copy and the host image (whose
 *      64-byte header carries the launch geometry).  The plan stays valid
 *      while the pointers it names do; it can be launched any number of
 *      times.
 * Problems must not write overlapping y ranges.  Errors: INVALID_ARG,
 * UNSUPPORTED, WORKSPACE, HIP. */
typedef struct {
  const uint32_t* w;
  const uint16_t* scales;
  const uint16_t* biases;
  const uint16_t* x;
  float* y;
  int32_t n;
  int32_t k;
} qmm_gemv_problem;

int qmm_qgemv_batched_plan(const qmm_gemv_problem* problems, int count, int bits,
                           int group_size, void* plan, size_t plan_bytes,
                           size_t* plan_bytes_needed);
int qmm_qgemv_batched(const void* plan_device, const void* plan_host, qmm_stream stream);

/* ----------------------------------------------------------- prefill GEMM
 * y[m, n] = sum_k x[m, k] * W_hat[n, k]   (BaseRT §3.4: tiled prefill GEMM)
 *   x [m, k] fp16 bits; y [m, n] fp32 (overwritten); other operands as GEMV.
 * Weight tiles are dequantized to fp16 in registers (one rounding of
 * s*q + b) and multiplied on the fp16 matrix cores with fp32 accumulation.
 * workspace may be NULL when qmm_qgemm_workspace_size returns 0.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, HIP. */
size_t qmm_qgemm_workspace_size(int m, int n, int k, int bits, int group_size);
int qmm_qgemm(const uint32_t* w, const uint16_t* scales, const uint16_t* biases,
              const uint16_t* x, float* y, int m, int n, int k, int bits, int group_size,
              void* workspace, size_t workspace_bytes, qmm_stream stream);

/* ---------------------------------------------------- batched prefill GEMM
 * Several independent y_p = x_p W_hat_p^T (same arithmetic as qmm_qgemm) in
 * ONE launch: e.g. the q, k and v projections of a layer, or gate and up,
 * whose tiles together fill the chip where each alone would not (BaseRT
 * §3.4 tiled prefill GEMM; §3 amortized dispatch).  Two steps, as for the
 * batched GEMV:
 *   1. qmm_qgemm_batched_plan (host only, no HIP call): from `count`
 *      problem descriptors (device pointers, host array) choose one tile
 *      shape and k-split count for the batch and write the plan image into
 *      host memory `plan` of `plan_bytes`.  *plan_bytes_needed receives the
 *      image size and *workspace_bytes_needed the device workspace size
 *      (0 when k is not split); if plan is NULL or too small the call
 *      returns QMM_ERR_WORKSPACE without writing the image.  Each problem
 *      has its own m >= 0, n >= 1 and k (a multiple of 64); all share bits
 *      and group_size.  A problem with m = 0 is skipped (its x and y may be
 *      NULL).
 *   2. Copy the image verbatim to device memory (16-byte aligned), then
 *      call qmm_qgemm_batched with the device copy, the host image and the
 *      workspace.
 * Workspace (contents on entry do not matter): with k split, each split
 * writes an fp32 partial tile there and a second, short kernel adds the
 * partials of every tile in split order, so results are identical from run
 * to run.  Calls that share a workspace must not run concurrently.
 * Problems must not write overlapping y ranges.
 * Weight layout: `bits` alone means every w is row-major [n, k*bits/32] as
 * everywhere else; `bits | QMM_WEIGHTS_TILED` means every w was produced by
 * qmm_repack_tiled (then every n must be a multiple of 32), which the
 * prefill tiles read with fewer, fully contiguous loads.  Scales and biases
 * are row-major unless `bits` also carries QMM_SCALES_TILED: then every
 * `scales` pointer is an interleaved scale-and-bias array produced by
 * qmm_repack_scales_tiled (16-byte aligned; `biases` is not read and may be
 * NULL), which needs QMM_WEIGHTS_TILED, group_size 64, 2- to 8-bit codes and
 * k a multiple of 256.  The two scale layouts give identical results.  The
 * flag is taken the same way by qmm_qgemm and by the grouped MoE calls
 * (qmm_qgemm_grouped, _noalloc, _routed and qmm_moe_gate_up_swiglu, whose
 * stacked expert scales [E, n, k/64] repack as one [E*n, k/64] array).
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, HIP. */
#define QMM_WEIGHTS_TILED 0x100
#define QMM_SCALES_TILED 0x200
typedef struct {
  const uint32_t* w;
  const uint16_t* scales;
  const uint16_t* biases;
  const uint16_t* x;
  float* y;
  int32_t m;
  int32_t n;
  int32_t k;
} qmm_gemm_problem;

int qmm_qgemm_batched_plan(const qmm_gemm_problem* problems, int count, int bits,
                           int group_size, void* plan, size_t plan_bytes,
                           size_t* plan_bytes_needed, size_t* workspace_bytes_needed);
int qmm_qgemm_batched(const void* plan_device, const void* plan_host, void* workspace,
                      size_t workspace_bytes, qmm_stream stream);

/* --------------------------------------------- mixture-of-experts grouped
 * BaseRT (native-Metal LLM inference on Apple Silicon), abstract and Fig. 1:
 * the mixture-of-experts prefill (Qwen3-30B-A3B, 4-bit) is where the pages
 * report their larger advantage; they give no mechanism, so the one here is
 * token-to-expert bucketing with one tile schedule per expert.  §3.3 applies
 * as for the GEMM (dequantization inside the inner loop).
 *
 * Pair p = t * top_k + j routes token t to expert e = expert_ids[t, j]:
 *     y[p, n] = sum_k A[row(p), k] * W_hat_e[n, k]
 *   w       [E, n, k*bits/32]; scales, biases [E, n, k/group_size]
 *   a       fp16 bits; a_row_per_pair = 0: A is [T, k] and row(p) = p / top_k
 *           (gate / up projections read the token); 1: A is [T*top_k, k] and
 *           row(p) = p (the down projection reads the pair's own row)
 *   expert_ids [T, top_k] int32, each in [0, E).  A pair whose id lies outside
 *           that range is not computed: its output row is NaN, and the count
 *           of such pairs is recorded in the plan header (below).
 *   y       [T*top_k, n] fp32 (overwritten)
 * Device-side token-to-expert bucketing (histogram, scan, scatter) builds
 * one tile list per expert in the workspace; the grouped GEMM then gathers
 * A rows, dequantizes that expert's weight tiles and scatters output rows.
 * The workspace size depends only on (T, top_k, E); n, k, bits and
 * group_size are accepted so that a caller can size it from the same
 * arguments as the product.
 *
 * Routing plan / workspace image (device memory, int32 words):
 *   word 0  row tiles in the list     word 1  rows per row tile
 *   word 2  pairs (T * top_k)         word 3  experts E
 *   word 4  pairs whose expert id was outside [0, E)  (byte offset 16)
 *   words 5..7 zero; then the bucketed pair list, the row-tile list and
 *   the per-chunk expert counts that the bucketing launches pass between them.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, HIP. */
size_t qmm_qgemm_grouped_workspace_size(int t, int top_k, int e, int n, int k, int bits,
                                        int group_size);
int qmm_qgemm_grouped(const uint32_t* w, const uint16_t* scales, const uint16_t* biases,
                      const uint16_t* a, int a_row_per_pair, const int32_t* expert_ids,
                      float* y, int t, int top_k, int e, int n, int k, int bits,
                      int group_size, void* workspace, size_t workspace_bytes,
                      qmm_stream stream);

/* Allocation-free grouped product, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc): qmm_qgemm_grouped with the same arguments minus the
 * workspace.  Its bucket lists and tile list live in a static device array
 * of QMM_GROUPED_SCRATCH_BYTES (1 MiB) that each GPU holds from the first
 * call on it until the process ends; the call allocates nothing, frees
 * nothing and calls no allocating library routine.  The scratch serves
 * every (t, top_k, e) whose qmm_qgemm_grouped_workspace_size is at most
 * 1 MiB (up to about 231,000 pairs, e.g. 28,900 tokens at top-8, with
 * E = 128); larger problems are refused with QMM_ERR_WORKSPACE before any
 * launch.  Every call on one GPU shares that GPU's array, so calls that
 * overlap on one GPU (several streams, several host threads) race and must
 * be serialized by the caller; the array is never cleared (each call
 * rewrites every word it reads).  Pairs with an out-of-range expert id get
 * NaN rows as in qmm_qgemm_grouped; their count stays in the scratch and is
 * not reported.  Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, HIP. */
#define QMM_GROUPED_SCRATCH_BYTES (1u << 20)
int qmm_qgemm_grouped_noalloc(const uint32_t* w, const uint16_t* scales, const uint16_t* biases,
                              const uint16_t* a, int a_row_per_pair, const int32_t* expert_ids,
                              float* y, int t, int top_k, int e, int n, int k, int bits,
                              int group_size, qmm_stream stream);

/* Routing plan shared by the grouped products of one MoE layer (BaseRT,
 * abstract and Fig. 1: MoE prefill; §3 amortized dispatch).  Gate, up and
 * down read the same expert ids, so the token-to-expert bucketing (the first
 * launch of qmm_qgemm_grouped) can run once:
 *   qmm_moe_route        buckets expert_ids [T, top_k] into `plan` (device
 *                        memory of qmm_moe_route_size(T, top_k, E) bytes,
 *                        16-byte aligned, caller-owned; contents on entry
 *                        do not matter);
 *   qmm_qgemm_grouped_routed  the grouped product of qmm_qgemm_grouped, with
 *                        the same arguments except that `plan` and its size
 *                        `plan_bytes` replace expert_ids and the workspace.
 * The plan stays valid while expert_ids is unchanged, for any n, k, bits and
 * group size, and may be read by several launches in flight.  plan_bytes
 * below qmm_moe_route_size(T, top_k, E) is refused on the host (WORKSPACE);
 * a plan built for another (T, top_k, E) or another row tile is detected on
 * the device and the whole output is then written as NaN.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, HIP. */
size_t qmm_moe_route_size(int t, int top_k, int e);
int qmm_moe_route(const int32_t* expert_ids, int t, int top_k, int e, void* plan,
                  size_t plan_bytes, qmm_stream stream);
int qmm_qgemm_grouped_routed(const uint32_t* w, const uint16_t* scales, const uint16_t* biases,
                             const uint16_t* a, int a_row_per_pair, const void* plan,
                             size_t plan_bytes, float* y, int t, int top_k, int e, int n, int k,
                             int bits, int group_size, qmm_stream stream);

/* Mixture-of-experts FFN block around the grouped products (BaseRT §3.3:
 * the FFN's matmuls and activation fused into fewer kernels; abstract and
 * Fig. 1: MoE prefill).
 *   qmm_moe_gate_up_swiglu  for every pair p (token row p / top_k of x
 *       [T, k] fp16), with e = the pair's expert from `plan` (qmm_moe_route,
 *       plan_bytes as for qmm_qgemm_grouped_routed):
 *           h[p, c] = fp16( silu(g) * u ),  silu(g) = g / (1 + exp(-g)),
 *           g = sum_k x[row, k] W_gate_e[c, k],  u = likewise with W_up_e
 *       (g, u and the SwiGLU in fp32; one rounding to fp16).  w_gate, w_up
 *       [E, n, k*bits/32] with their scales and biases as in
 *       qmm_qgemm_grouped; h [T*top_k, n] fp16 bits (overwritten) is the
 *       down projection's A (a_row_per_pair = 1).  bits = 16: fp16 weights.
 *       Rows of pairs with an out-of-range expert id, and all of h when the
 *       plan was built for other counts, are written as fp16 NaN.
 *   qmm_moe_combine  y[t, c] = sum_{j < top_k} weights[t, j] * y_pairs[t*top_k + j, c]
 *       with the slots added in order j = 0, 1, ... (fp32 fma), so the result
 *       does not depend on scheduling.  y_pairs [T*top_k, n] fp32 (the down
 *       projection's output), weights [T, top_k] fp32, y [T, n] fp32.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE (plan too small), HIP. */
int qmm_moe_gate_up_swiglu(const uint32_t* w_gate, const uint16_t* s_gate, const uint16_t* b_gate,
                           const uint32_t* w_up, const uint16_t* s_up, const uint16_t* b_up,
                           const uint16_t* x, const void* plan, size_t plan_bytes, uint16_t* h,
                           int t, int top_k, int e, int n, int k, int bits, int group_size,
                           qmm_stream stream);
int qmm_moe_combine(const float* y_pairs, const float* weights, float* y, int t, int top_k, int n,
                    qmm_stream stream);

/* Routing to experts: the step before qmm_moe_route and qmm_moe_combine.
 * From router logits [T, E] fp32 (e.g. the output of qmm_qgemm over the
 * router's weights), for every token t:
 *   s[e] = softmax over e of logits[t, e]       (QMM_SCORE_SOFTMAX)
 *        = 1 / (1 + exp(-logits[t, e]))         (QMM_SCORE_SIGMOID)
 *   c[e] = s[e] + bias[e]                       (bias [E] fp32 or NULL)
 *   the E experts form `groups` groups of E / groups neighbours; a group's
 *       score is the sum of its group_top (1 or 2) largest c, and the
 *       group_keep groups of the largest scores stay
 *   expert_ids[t, :] = the top_k experts of those groups by c, largest first
 *   weights[t, j] = scale * s[id_j] / (renormalize ? sum_j s[id_j] : 1)
 * Equal values go to the lower index, of groups and of experts.  Where only the
 * order of the scores counts (no bias, group_top = 1) logits are compared as
 * they are; otherwise the choice is that of the formulas in 64 bits (where
 * sigmoid scores of logits from 37 on are 1 and equal).  The bias moves the
 * choice, never the weights, which are formed in 64 bits and rounded once.
 * A logit of -inf is an expert switched off: its score is 0 (it can still be
 * returned, with weight 0, where top_k experts cannot be had otherwise or a
 * bias lifts it).  A renormalizing sum of 0 (every chosen expert switched off,
 * or of a sigmoid logit below -745, 0 in 64 bits) gives weights 0.  A token whose scores, choices or group scores hold
 * a NaN (a NaN logit or bias; +inf under softmax) gets expert_ids
 * 0 .. top_k-1 and NaN weights, so that the failure shows in its output.
 *   groups: divides E, at most 64 (1: no groups, then group_keep = 1);
 *   top_k: at most 64 and at most the experts of group_keep groups;
 *   E at most 1024; T below 2^26.
 * One launch (of 2^26 - 3 tokens and more it can be two), no workspace.  t = 0
 * does nothing.
 * Errors: INVALID_ARG, UNSUPPORTED (score), HIP. */
#define QMM_SCORE_SOFTMAX 0
#define QMM_SCORE_SIGMOID 1
int qmm_moe_topk(const float* logits, const float* bias, int32_t* expert_ids, float* weights, int t,
                 int e, int top_k, int score, int groups, int group_keep, int group_top,
                 int renormalize, float scale, qmm_stream stream);

/* ----------------------------------------- low-rank adapters per request
 * Many requests share a projection (qmm_qgemv, qmm_qgemm, the batched and
 * the grouped products) and each has a low-rank adapter of its own:
 *   y[p, :] = base[p, :] + scales[i] * B_s (A_s x[row(p), :]),   i = adapter_ids[p / top_k]
 * for the rows p < t * top_k.
 *   Dense projections: experts = 0, expert_ids NULL, top_k = 1; s = i.
 *   Experts' products of a routed layer: pair p = token * top_k + j has
 *       s = i * experts + expert_ids[p], the ids of qmm_moe_topk or
 *       qmm_moe_route's input; row(p) = p with x_row_per_pair = 1 (the down
 *       projection), p / top_k with 0 (gate, up).
 *   x     fp16 bits, [t, k] or, with x_row_per_pair, [t * top_k, k]
 *   a     fp16 bits, [adapters (x experts), rank, k]
 *   b     fp16 bits, [adapters (x experts), n, rank]
 *   base  fp32 [t * top_k, n], the shared product; it may be y itself (added
 *         in place) or NULL (y is the adapters' part alone), but must not
 *         overlap y otherwise
 *   y     fp32 [t * top_k, n], overwritten; must not overlap x
 *   adapter_ids  [t] int32; -1: no adapter, the row is base (0 without base)
 *   scales       [adapters] fp32 (alpha / rank), or NULL for 1
 * An adapter id below -1 or >= adapters, or an expert id outside
 * [0, experts) of a row with an adapter, makes the row NaN.
 * The up to 8 problems of one call (q, k and v; gate and up) share the ids and
 * run in the same launches: no y may overlap another problem's y, base or x
 * (two adapters on one output are two calls).  Adapters of smaller
 * rank are padded with zeros to the problem's rank, a multiple of 8 up to
 * 256; k is a multiple of 64 up to 2^24, adapters x experts at most 4096, n at most
 * 2097152, t * top_k at most 2^27.  Both products are sums of exact fp16 products in fp32; on the
 * matrix cores the sum A x enters the second one as two fp16, off by up to 2^-23
 * of the row's largest value of it.  Non-finite adapter weights make
 * non-finite outputs.  Results do not depend on scheduling, nor on what the
 * other rows hold.
 * Workspace: qmm_lora_workspace_size bytes for `rows` = t * top_k and `slots` =
 * adapters * max(1, experts) (only k and rank of the problems are read; 0 for
 * sizes that are refused), 16-byte aligned, contents on entry do not matter;
 * calls (and captured graphs) that share one must not run concurrently.
 * One to four launches, by the sizes alone.
 * t = 0 does nothing.
 * Errors: INVALID_ARG, WORKSPACE, HIP. */
typedef struct {
  const uint16_t* x;
  const uint16_t* a;
  const uint16_t* b;
  const float* base;
  float* y;
  int32_t n;
  int32_t k;
  int32_t rank;
  int32_t x_row_per_pair;
} qmm_lora_problem;

size_t qmm_lora_workspace_size(const qmm_lora_problem* problems, int count, int rows, int slots);
int qmm_lora(const qmm_lora_problem* problems, int count, const int32_t* adapter_ids,
             const int32_t* expert_ids, const float* scales, int t, int top_k, int adapters,
             int experts, void* workspace, size_t workspace_bytes, qmm_stream stream);

/* -------------------------------------------------- products in 8-bit integers
 * Both operands are 8-bit integers with one fp32 scale a row: w [n, k] a scale
 * for each output channel, x [m, k] a scale for each token.
 *   s[r]    = fp32( max_k |x[r, k]| / 127 )
 *   q[r, k] = rint( x[r, k] / s[r] )     (the exact quotient, ties to even)
 *   y[m, n] = s_x[m] s_w[n] sum_k q_x[m, k] q_w[n, k]  (+ bias[n])
 * qmm_i8_quantize gives codes and scales of rows: of a weight matrix at load
 * time (a row is an output channel), of activations (a row is a token).  The
 * products also take x in 16 or 32 bits and round its rows themselves, to the
 * same codes.  The sum is an exact int32; it is rounded to fp32, multiplied by
 * the two scales and rounded after each (then once more to a 16-bit y), so a
 * result depends on nothing but its own row, column and scales.
 * A row whose largest magnitude is below 2^-119 has scale 0 and codes 0; a row
 * that holds a NaN or an infinity has scale NaN and codes 0, and so a row of
 * NaN in y.  Given codes may be anything from -128 to 127.
 *   types  QMM_F32, QMM_F16, QMM_BF16 (bit patterns); QMM_I8: codes, with their scales
 *   sizes  k a multiple of 16 up to 131008; n in [1, 2097152]; m in [0, 16777215],
 *          also over all problems of a call; the outputs of a call at most 2^35
 *   w, x, codes and workspaces 16-byte aligned, scales and bias 4-byte, y by
 *   its type (on 16 bytes, with n a multiple of 4, it is stored by whole pieces)
 * Errors of all: INVALID_ARG, UNSUPPORTED (type), WORKSPACE, HIP. */
#define QMM_F32 0
#define QMM_F16 1
#define QMM_BF16 2
#define QMM_I8 3

/* codes [m, k], scales [m] of x [m, k] (x_type: QMM_F32, QMM_F16 or QMM_BF16).
 * One launch; codes and scales must not overlap x or each other. */
int qmm_i8_quantize(const void* x, int x_type, int8_t* codes, float* scales, int m, int k,
                    qmm_stream stream);

/* Up to 8 products of one call (q, k and v; gate and up; or one alone) run
 * together.  Problems that name the same x (with the same m, k and type) have it
 * rounded once.  No y may overlap another problem's y, or any operand.
 *   x_scales  [m] with x_type QMM_I8, NULL otherwise
 *   bias      [n] fp32 or NULL
 * Workspace: qmm_i8_gemm_workspace_size bytes (x, m, n, k and x_type of the
 * problems are read; 0 for sizes that are refused, and where none is needed:
 * then it may be NULL), contents on entry do not matter; it must not overlap an
 * operand or an output; calls (and captured graphs) that share one must not run
 * concurrently.  m = 0: the problem does
 * nothing.  One to three launches, by sizes (one more for each further type of x). */
typedef struct {
  const int8_t* w;
  const float* w_scales;
  const void* x;
  const float* x_scales;
  const float* bias;
  void* y;
  int32_t m;
  int32_t n;
  int32_t k;
  int32_t x_type;
  int32_t y_type;
} qmm_i8_problem;

size_t qmm_i8_gemm_workspace_size(const qmm_i8_problem* problems, int count);
int qmm_i8_gemm(const qmm_i8_problem* problems, int count, void* workspace, size_t workspace_bytes,
                qmm_stream stream);

/* The experts' products of a routed layer, from a plan of qmm_moe_route for the
 * same (t, top_k, e): pairs, rows and out-of-range experts (NaN rows) as in
 * qmm_qgemm_grouped_routed; a plan built for other counts makes the whole
 * output NaN.  The output must not overlap any operand, nor the plan.
 *   qmm_i8_gemm_grouped  y[p, :] = the product of row(p) of a with w [E, n, k] of
 *       the pair's expert, w_scales [E, n]; y [t * top_k, n] of y_type
 *   qmm_i8_moe_gate_up_swiglu  h[p, :] = silu(g) u with g and u the products of
 *       x's row p / top_k with w_gate and w_up [E, n, k] of the pair's expert
 *       (fp32 until h, of h_type, is rounded)
 *   a, x  of a_type / x_type; with QMM_I8 its scales, one for each row, NULL
 *         otherwise.  rows * k must be below 2^32, and the tiles of a call (64 rows
 *         of an expert by 128 columns or more each) about 2^23 at most.
 * Workspace: qmm_i8_grouped_workspace_size bytes for the rows of a or x (0 with
 * QMM_I8: then it may be NULL), as above. */
size_t qmm_i8_grouped_workspace_size(int rows, int k, int x_type);
int qmm_i8_gemm_grouped(const int8_t* w, const float* w_scales, const void* a, const float* a_scales,
                        int a_type, int a_row_per_pair, const void* plan, size_t plan_bytes, void* y,
                        int y_type, int t, int top_k, int e, int n, int k, void* workspace,
                        size_t workspace_bytes, qmm_stream stream);
int qmm_i8_moe_gate_up_swiglu(const int8_t* w_gate, const float* s_gate, const int8_t* w_up,
                              const float* s_up, const void* x, const float* x_scales, int x_type,
                              const void* plan, size_t plan_bytes, void* h, int h_type, int t, int top_k,
                              int e, int n, int k, void* workspace, size_t workspace_bytes,
                              qmm_stream stream);

/* ------------------------------------------------ load-time quantization
 * Asymmetric min/max quantization of a dense fp32 weight W[n, k] into the
 * packed format above: per group, s = fp16((max - min) / L) and
 * b = fp16(min) with L = 2^bits - 1 (fp32 arithmetic, IEEE division,
 * round-to-nearest-even), q = clamp(rint((w - b) / s), 0, L), and q = 0 for
 * every element when s == 0.  Work done once when a model is loaded
 * (BaseRT §3.2 prepares everything at load time).
 *   w_f32 [n, k] fp32; words [n, k*bits/32]; scales, biases [n, k/gs] fp16 bits.
 * Errors: INVALID_ARG, UNSUPPORTED, HIP. */
int qmm_quantize(const float* w_f32, uint32_t* words, uint16_t* scales, uint16_t* biases,
                 int n, int k, int bits, int group_size, qmm_stream stream);

/* bf16 weights (load time).  The matrix cores multiply fp16 by fp16 or bf16
 * by bf16, not fp16 activations by bf16 weights, so bf16 weights are
 * converted once to fp16 and then used as bits = 16:
 *   dst[i] = fp16(bf16 src[i]), round to nearest even; exact for every bf16
 *   whose magnitude lies in fp16's normal range, +-inf beyond 65504.
 *   src, dst: count uint16 bit patterns (count even, 4-byte aligned; dst may
 *   equal src for an in-place conversion).
 * Errors: INVALID_ARG, HIP. */
int qmm_convert_bf16(const uint16_t* src, uint16_t* dst, size_t count, qmm_stream stream);

/* Tile-interleaved weights for the batched prefill GEMM (load time; a
 * layout of this library's own, not from the pages): out holds the same
 * words as the row-major w [n, k*bits/32], each 64-code group moved whole:
 *   group g of column c: w word (c * G + g) * WPG
 *                     -> out word ((c / 32) * G * 32 + g * 32 + c % 32) * WPG
 *   with G = k / 64 and WPG = 2 * bits words per group (32 for bits = 16),
 * so the 32 columns of one matrix-core column block are contiguous for each
 * group.  n must be a multiple of 32 and k of 64; w and out are device
 * buffers of n * k * bits / 8 bytes (16-byte aligned, not overlapping); out
 * is used with QMM_WEIGHTS_TILED: on the bits of qmm_qgemm, of a batched
 * plan, of qmm_qgemm_grouped, qmm_qgemm_grouped_routed and
 * qmm_moe_gate_up_swiglu (stacked experts [E, n, ...] repack as one
 * [E*n, ...] matrix, which keeps each expert's block whole when n is a
 * multiple of 32).  The decode GEMV keeps reading row-major weights.
 * Errors: INVALID_ARG, UNSUPPORTED, HIP. */
int qmm_repack_tiled(const uint32_t* w, uint32_t* out, int n, int k, int bits, qmm_stream stream);

/* Interleaved scales and biases for the prefill GEMM over tile-interleaved
 * weights (load time; a layout of this library's own, not from the pages):
 * out holds every scale and bias of the row-major scales and biases
 * [n, k/64] (groups of 64 codes), for each block of 32 columns and each
 * quad of 4 groups the 32 columns' 16-byte {s[4q .. 4q+3], b[4q .. 4q+3]}
 * next to each other:
 *   scales[c * G + g] -> out[((c / 32) * (G / 4) * 32 + c % 32) * 8 + (g / 4) * 256 + g % 4]
 *   biases[c * G + g] -> the same index + 4,      with G = k / 64,
 * so one wave's scale loads read whole lines.  n must be a multiple of 32 and
 * k of 256; scales and biases are device arrays of n * k / 64 fp16 (2-byte
 * aligned), out one of 2 * n * k / 64 fp16 (16-byte aligned, overlapping
 * neither); out is used as `scales` with QMM_SCALES_TILED (stacked MoE expert
 * scales and biases [E, n, k/64] repack as one [E*n, k/64] matrix, which
 * keeps each expert's block whole when n is a multiple of 32).
 * Errors: INVALID_ARG, HIP. */
int qmm_repack_scales_tiled(const uint16_t* scales, const uint16_t* biases, uint16_t* out, int n, int k,
                            qmm_stream stream);

/* ------------------------------------------------------------- diagnostics
 * Expose the device-side stages of the hot path for bit-exact checking.
 * qmm_unpack_codes: codes[n, k] (uint8) = the codes of `w`, decoded with
 *   the same register unpack the GEMV and GEMM kernels use.
 * qmm_dequant: out[n, k] = W_hat as fp32 (out_is_f16 = 0; one rounding of
 *   the exact s*q + b) or as fp16 bits (out_is_f16 = 1; one rounding, the
 *   value the GEMM feeds to the matrix cores).
 * Errors: INVALID_ARG, UNSUPPORTED, HIP. */
int qmm_unpack_codes(const uint32_t* w, uint8_t* codes, int n, int k, int bits,
                     qmm_stream stream);
int qmm_dequant(const uint32_t* w, const uint16_t* scales, const uint16_t* biases,
                void* out, int out_is_f16, int n, int k, int bits, int group_size,
                qmm_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* QMM_H */
