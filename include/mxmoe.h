/*
 * mxmoe.h -- C ABI of libmxmoe.so, the GB300 (sm_103a) MX block-scaled
 * sparse-MoE expert layer.
 *
 * The layer (one MoE block of a transformer) computes, for T tokens of hidden
 * size H, E routed experts with intermediate size I and top-k routing, plus one
 * shared expert folded into the expert table at index E as an always-selected
 * expert of weight 1:
 *
 *   act      = MXFP8(x)                                   mx_quantize_act
 *   ids, w   = top-k(logits), softmax over the k chosen    moe_route_topk
 *   slots    = tokens grouped by expert                   moe_permute
 *   h[s]     = MXFP8( silu(act[t].Wg[e]) * (act[t].Wu[e]) ) moe_grouped_gemm_swiglu
 *   out[t]  += w[s] * (h[s] . Wd[e])                      moe_grouped_gemm_down_combine
 *
 * Sources: the MX weight formats and the shared-expert folding follow
 * "Tracing the bottleneck: optimising MiniMax M3 on AMD Instinct MI355X"
 * (opening results list for MXFP8/MXFP4 weights; Figure 4 for the shared
 * expert placed in the routed table and selected for every token; Figure 3 and
 * the surrounding passage for separate small-M / large-M schedules; the
 * passage after Figure 4 for moving weight/scale re-layout to load time).  The
 * combine fused into the down projection's epilogue follows "Kimi K3
 * performance in vLLM: 2.8x throughput" (section on fusing the MXFP4 top-k
 * finalize into the epilogue).  The element formats are those of the OCP
 * Microscaling Formats (MX) v1.0 specification.
 *
 * Conventions for every call
 *  - Pointers are DEVICE pointers owned by the caller unless stated; the
 *    library never allocates and never synchronises the stream.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls are
 *    asynchronous: they validate arguments on the host, enqueue kernels and
 *    return.  A return of MX_OK means the work was enqueued.
 *  - Device-side errors (a bounded wait that ran out, an expert id out of
 *    range) are OR-ed into a status word at the start of the caller's
 *    workspace; read and clear it with moe_get_status.
 *  - Workspaces must be zero-filled once before their first use (the library
 *    leaves them ready for the next call of the same function, of any size that
 *    they are large enough for).
 *  - Formats: MX_E4M3 (MXFP8, one byte per element) and MX_E2M1 (MXFP4, two
 *    elements per byte, element 2i in the low nibble).  Every 32 consecutive
 *    elements along K share one E8M0 scale byte (value 2^(code-127)).
 *  - Non-finite inputs are a precondition violation: results are unspecified.
 */
#ifndef MXMOE_H_
#define MXMOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* mx_stream_t; /* same type as cudaStream_t */

#if defined(__GNUC__)
#define MX_API __attribute__((visibility("default")))
#else
#define MX_API
#endif

/* ---- status codes ---- */
#define MX_OK 0
#define MX_ERR_INVALID_ARG 1  /* null pointer, non-positive size, k > E, k > 32 ... */
#define MX_ERR_UNSUPPORTED 2  /* shape the kernels do not handle (see each call) */
#define MX_ERR_ALIGNMENT 3    /* a pointer is not 16-byte (weights: 256-byte) aligned */
#define MX_ERR_WORKSPACE 4    /* workspace / destination smaller than required */
#define MX_ERR_CUDA 5         /* a CUDA runtime/driver call or kernel launch failed */
#define MX_ERR_TIMEOUT 6      /* device status: a bounded wait inside a kernel ran out */
#define MX_ERR_DEVICE_ARG 7   /* device status: an expert id or slot id out of range */

/* ---- element formats ---- */
#define MX_E4M3 0
#define MX_E2M1 1

/* Human-readable name of a status code (static string, never NULL). */
MX_API const char* mx_status_string(int status);

/* Activation quantisation, bf16 -> MXFP8 (E4M3 codes + E8M0 scales).
 *   x_bf16  [T, H] row-major bf16.  codes [T, H] bytes.  scales [T, H/32] bytes.
 * Per row and per block of 32 along H: shared exponent
 * s = clamp(floor(log2(amax)) - 8, -127, 127) (an all-zero block gives -127),
 * scale byte s + 127, element code = E4M3 value of x / 2^s rounded to nearest
 * even and saturated to +-448; a negative value that rounds to zero keeps its
 * sign (0x80).  Bit-exact with the reference definition.
 * Errors: MX_ERR_INVALID_ARG (null, T < 0, H <= 0), MX_ERR_UNSUPPORTED
 * (H % 32), MX_ERR_ALIGNMENT (x or codes not 16-byte aligned).
 * Source: the MI355X page (opening results list: MXFP8 and MXFP4 models;
 * the passage on the native MXFP8 linear backend); the element and scale rule
 * is that of OCP MX v1.0. */
MX_API int mx_quantize_act(const void* x_bf16, int T, int H, uint8_t* codes, uint8_t* scales,
                    mx_stream_t stream);

/* mx_quantize_act to a chosen MX format: fmt MX_E4M3 (as mx_quantize_act) or
 * MX_E2M1 (MXFP4: emax 2, codes [T, H/2] bytes, element 2i in the low nibble,
 * saturation at 6), scales [T, H/32].  Errors as mx_quantize_act, plus
 * MX_ERR_INVALID_ARG for another fmt.  Source: as mx_quantize_act; MXFP4
 * activations are the mx_layer_opts act_fmt variant. */
MX_API int mx_quantize_act_ex(const void* x_bf16, int T, int H, int fmt, uint8_t* codes, uint8_t* scales,
                              mx_stream_t stream);

/* Weight quantisation, fp32 -> MXFP8 or MXFP4 (load-time helper; same rule as
 * mx_quantize_act with emax 8 for E4M3 and 2 for E2M1, saturation at 6 for
 * E2M1).  w [rows, K] fp32; codes [rows, K] (E4M3) or [rows, K/2] (E2M1);
 * scales [rows, K/32].  Errors as mx_quantize_act (K % 32). */
MX_API int mx_quantize_weights(const float* w, int64_t rows, int K, int fmt, uint8_t* codes,
                        uint8_t* scales, mx_stream_t stream);

/* Router: per token, the k largest of E fp32 logits, ties to the lowest expert
 * index, in descending logit order, and their softmax (over the k selected).
 *   logits [T, E] fp32; topk_ids [T, k] int32; topk_w [T, k] fp32.
 * Ids are bit-exact with the reference; weights are fp32 (a few ulp).
 * Errors: MX_ERR_INVALID_ARG (null, T < 0, E <= 0, k < 1, k > E, k > 32),
 * MX_ERR_UNSUPPORTED (E > 1024).
 * Source: the MI355X page, Figure 4 and its passage (each token's routed
 * experts, with the shared expert added as a slot every token selects) and the
 * correctness passage (the expert mask a token is routed through must be
 * exact); the Kimi K3 page, section on the MXFP4 top-k finalize.  The pages fix
 * no tie rule: lowest index first is this library's reading. */
MX_API int moe_route_topk(const float* logits, int T, int E, int k, int32_t* topk_ids, float* topk_w,
                   mx_stream_t stream);

/* Router GEMM with top-k in its epilogue (the step ahead of moe_route_topk):
 *   logits[t, e] = sum_h x[t, h] * w_router[e, h]   (bf16 inputs, fp32 accumulation;
 *     products of bf16 values are exact in fp32)
 *   topk_ids[t, :] = the k experts with the largest score logit + bias[e]
 *     (one fp32 addition), lowest index on ties, descending score order
 *   topk_w[t, :] = softmax of the chosen experts' unbiased logits (fp32).
 *   x_bf16 [T, H], w_router_bf16 [E, H] row-major, 16-byte aligned.
 *   bias [E] fp32 or NULL (no bias): a load-balancing bias that steers which
 *     experts are chosen but not their weights (this library's reading; the
 *     pages give no router).  logits [T, E] or NULL.  topk_ids and topk_w
 *     both NULL: logits only (then logits must be given).
 *   ws: a 256-byte-aligned workspace of at least 256 bytes, zero-filled once;
 *     its first word is the status word moe_get_status reads, its second a
 *     counter of the small-batch kernel.
 * Up to 128 tokens with somewhere to keep the logits (logits given, or ws of
 * at least 256 + 4*T*E bytes) run a CUDA-core kernel over blocks of 2 experts
 * (the router is then a weight-streaming matrix-vector product) whose last
 * block selects; larger batches run the tensor-core GEMM with the selection
 * in its epilogue.  Both sum the same exact bf16 products in fp32 (in
 * different orders).
 * Errors: MX_ERR_INVALID_ARG, MX_ERR_UNSUPPORTED (H % 64, E > 512, k > 16),
 * MX_ERR_ALIGNMENT, MX_ERR_WORKSPACE.
 * Source: the MI355X page, Figure 4 and its passage (tokens are routed to
 * experts by router scores; the router itself is not printed). */
MX_API int moe_route_gemm_topk(const void* x_bf16, const void* w_router_bf16, const float* bias, int T, int H,
                               int E, int k, float* logits, int32_t* topk_ids, float* topk_w, void* ws,
                               size_t ws_bytes, mx_stream_t stream);

/* Bytes of workspace moe_permute needs. */
MX_API size_t moe_permute_workspace_size(int T, int E, int k);

/* Token -> expert permutation with the shared expert folded in.
 *   counts [E+1]: tokens per expert, counts[E] = T (shared expert).
 *   offsets [E+2]: exclusive prefix of counts, offsets[E+1] = T*(k+1).
 *   sorted_slot [T*(k+1)]: slot ids t*(k+1)+j (j = k is the shared slot),
 *     grouped by expert ascending (shared last), tokens ascending inside each
 *     expert.  Bit-exact, deterministic, no host synchronisation.
 * topk_ids must hold k distinct ids in [0, E) per token; an id out of range
 * sets MX_ERR_DEVICE_ARG in the workspace status and is skipped.
 * Errors: MX_ERR_INVALID_ARG, MX_ERR_UNSUPPORTED (E > 1024),
 * MX_ERR_WORKSPACE (ws_bytes < moe_permute_workspace_size).
 * Source: the MI355X page, Figure 3 and its passage (the routed token count of
 * each expert is that expert's local M; grouped MoE programs are ordered so
 * that neighbours reuse activation rows and expert weight tiles) and Figure 4
 * (the shared expert sits in the routed table and the grouped GEMMs process it
 * in the same pass).  Expert-major, token-ascending order is this library's
 * reading, chosen so the result is unique. */
MX_API int moe_permute(const int32_t* topk_ids, int T, int E, int k, int32_t* counts, int32_t* offsets,
                int32_t* sorted_slot, void* ws, size_t ws_bytes, mx_stream_t stream);

/* moe_permute without a caller workspace.  The pages have no counterpart:
 * this entry exists for callers that are not allowed to allocate device
 * memory (for example a plugin whose host framework owns all device memory
 * and forbids cudaMalloc in its enqueue path, or a serving loop that must not
 * call cudaMalloc because it can synchronise the device).  It computes exactly
 * what moe_permute computes, using a fixed 400 KiB scratch array inside the
 * library that every GPU loading the library keeps until the process exits.
 *  - Limit: the scratch moe_permute_workspace_size(T, E, k) reports must fit
 *    in 400 KiB (T <= 8192, E <= 512, k <= 8 always fits); larger requests
 *    return MX_ERR_WORKSPACE and enqueue nothing.
 *  - The array is shared by every call on a device and keeps the last call's
 *    contents; calls that overlap on the GPU race, so keep them on one stream.
 *  - The first call on a device looks up the array's device address; make it
 *    before any stream capture.  The address is kept per device and CUDA
 *    context: after cudaDeviceReset the next call looks it up again.
 *    Device-side id errors are not reported.
 *  - Allocates nothing: no cudaMalloc/cudaFree or allocating library call. */
MX_API int moe_permute_no_alloc(const int32_t* topk_ids, int T, int E, int k, int32_t* counts,
                                int32_t* offsets, int32_t* sorted_slot, mx_stream_t stream);

/* Bytes of a prepared (kernel-layout) weight table.  which = 1: W1, the
 * gate/up projection [E1][2I][H] (rows 0..I-1 gate, I..2I-1 up); which = 2:
 * W2, the down projection [E1][H][I].  E1 = E + 1 experts (shared last). */
MX_API size_t moe_prepared_weight_bytes(int E1, int H, int I, int fmt, int which);

/* Load-time re-layout of a canonical MX weight table into the kernel layout
 * (done once per weight set, off the serving path).
 *   codes  [E1][rows][K] (E4M3) or [E1][rows][K/2] (E2M1), scales [E1][rows][K/32],
 *   rows/K = 2I/H for which = 1 and H/I for which = 2.
 *   dst: moe_prepared_weight_bytes(...) bytes, 256-byte aligned.
 * Errors: MX_ERR_INVALID_ARG, MX_ERR_UNSUPPORTED (H or I not a multiple of
 * 128), MX_ERR_ALIGNMENT, MX_ERR_WORKSPACE (dst_bytes too small).
 * Source: the MI355X page, the passage after Figure 4 (MXFP8 weight and scale
 * re-layout moved to model load; serving uses the prepared form directly). */
MX_API int moe_prepare_weights(const uint8_t* codes, const uint8_t* scales, int E1, int H, int I, int fmt,
                        int which, void* dst, size_t dst_bytes, mx_stream_t stream);

/* Bytes of workspace the two grouped GEMM calls need. */
MX_API size_t moe_gemm_workspace_size(int T, int H, int I, int E, int k);

/* Grouped gate/up GEMM with SwiGLU and MXFP8 re-quantisation of h fused into
 * the epilogue.  For every slot position p (expert e = the segment of
 * `offsets` holding p, token t = sorted_slot[p] / (k+1)):
 *   g_i = sum_h act[t,h] Wg[e,i,h],  u_i = sum_h act[t,h] Wu[e,i,h]  (fp32 accumulation
 *   of exactly decoded MX products), h_i = silu(g_i) * u_i, then h quantised
 *   per 32 along I exactly as mx_quantize_act does.
 *   act_codes/act_scales: MXFP8 activations [T, H], [T, H/32].
 *   offsets/sorted_slot: moe_permute output.  w1_prep: moe_prepare_weights(which=1).
 *   h_codes [T*(k+1), I], h_scales [T*(k+1), I/32]: row p = slot position p.
 * fp32 accumulation means an h code next to a rounding boundary may differ by
 * one step from an exact-arithmetic reference.
 * Errors: MX_ERR_INVALID_ARG, MX_ERR_UNSUPPORTED (H or I % 128, E > 1024),
 * MX_ERR_ALIGNMENT, MX_ERR_WORKSPACE, MX_ERR_CUDA.
 * Source: the MI355X page, Figure 3 and its passage (separate small-M and
 * large-M launchers, tiles chosen from the local shape, grouped programs
 * reordered for cache reuse), Figure 4 (routed and shared experts in one
 * grouped GEMM) and the correctness passage (packed gate/up slices, SwiGLU). */
MX_API int moe_grouped_gemm_swiglu(const uint8_t* act_codes, const uint8_t* act_scales,
                            const int32_t* offsets, const int32_t* sorted_slot, const void* w1_prep,
                            int fmt, int T, int H, int I, int E, int k, uint8_t* h_codes,
                            uint8_t* h_scales, void* ws, size_t ws_bytes, mx_stream_t stream);

/* Grouped down GEMM with the weighted scatter-combine fused into the epilogue:
 *   out[t, :] += w_s * sum_i h[p,i] Wd[e,:,i]   (w_s = topk_w[t,j] for a routed
 *   slot, 1 for the shared slot), fp32 atomic adds into `out`.
 *   out [T, H] fp32 must be zero-filled (or hold a residual) by the caller.
 * Errors: as moe_grouped_gemm_swiglu.
 * Source: the Kimi K3 page, section on moving the MXFP4 top-k finalize into
 * the epilogue (one launch and one intermediate write/read removed); the
 * MI355X page, Figure 4 (the shared expert's output added with the routed
 * ones). */
MX_API int moe_grouped_gemm_down_combine(const uint8_t* h_codes, const uint8_t* h_scales,
                                  const int32_t* offsets, const int32_t* sorted_slot,
                                  const float* topk_w, const void* w2_prep, int fmt, int T, int H,
                                  int I, int E, int k, float* out, void* ws, size_t ws_bytes,
                                  mx_stream_t stream);


/* Bytes of workspace moe_forward needs (intermediates + GEMM scratch). */
MX_API size_t moe_workspace_size(int T, int H, int I, int E, int k, int fmt);

/* The whole layer in one call, no host synchronisation: quantise, route,
 * permute, both grouped GEMMs; out [T, H] fp32 is overwritten.  Three kernel
 * launches: a prologue (routing, quantisation, zeroing of out, the
 * permutation and, on the wide schedule, the activation rows in slot order;
 * for more than 256 tokens its phases are separated by grid barriers, plus
 * two 4-byte memsets of its counters) and the two grouped GEMMs (up to 256
 * tokens as programmatically dependent launches).  A batch whose prologue grid
 * would not fit on the GPU at once falls back to separate permutation launches.
 * Errors: union of the step calls.
 * Source: the MI355X page, the passage on launch cost and graph execution and
 * Figure 4's passage (removing launches and intermediate traffic raised output
 * throughput most at concurrency 1); the Ling-3.0-flash page, on kernel nodes
 * of 1.5-6 us each whose launch floor is comparable to their arithmetic. */
MX_API int moe_forward(const void* x_bf16, const float* logits, const void* w1_prep, const void* w2_prep,
                int fmt, int T, int H, int I, int E, int k, float* out, void* ws, size_t ws_bytes,
                mx_stream_t stream);

/* Number of kernel launches moe_forward enqueues for this shape on the
 * current device (host only: no kernel runs; -1 for a shape moe_forward
 * rejects, 0 for T = 0). */
MX_API int moe_forward_launches(int T, int H, int I, int E, int k, int fmt);

/* ---- layer variants ---- */
#define MX_ACT_SWIGLU 0      /* h = silu(g) * u */
#define MX_ACT_SWIGLU_OAI 1  /* h = g' * sigmoid(alpha * g') * (u' + 1), g' = min(g, limit), u' = clamp(u, +-limit) */
#define MX_SHARED_FOLDED 0   /* shared expert as a routed-table slot every token selects */
#define MX_SHARED_DENSE 1    /* shared expert as its own dense MLP launches */

/* Options of the layer variants (a NULL pointer means the defaults: SwiGLU,
 * folded shared expert, MXFP8 activations).
 *  - activation: MX_ACT_SWIGLU or MX_ACT_SWIGLU_OAI.  SwiGLU-OAI follows the
 *    MI355X page's correctness passage (the model's SwiGLU-OAI parameters are
 *    passed into the MoE); the page gives no values, the caller does: alpha
 *    (the sigmoid slope) and limit (> 0; the gate is clamped above at limit,
 *    the up projection to [-limit, limit]).
 *  - shared_expert: MX_SHARED_FOLDED (the MI355X page's Figure 4: one grouped
 *    GEMM pair covers routed and shared experts) or MX_SHARED_DENSE (the path
 *    that figure replaces: the shared expert runs as its own dense gate/up and
 *    down launches after the routed ones; same arithmetic, two more launches).
 *  - act_fmt: MX_E4M3 (MXFP8 activations and h) or MX_E2M1 (MXFP4
 *    activations and h: x and h are quantised to E2M1 with an E8M0 scale per
 *    32 elements, emax 2, and both grouped GEMMs run on the packed-FP4 MMA
 *    with MXFP4 weights on both sides).  MX_E2M1 needs fmt == MX_E2M1
 *    (MX_ERR_UNSUPPORTED with MXFP8 weights).  The activation codes
 *    (and h codes) are then [rows, K/2] bytes, element 2i in the low nibble.
 *    Source: the MI355X page's opening results list (an MXFP4 model) and its
 *    passage on native MX back ends; the element and scale rule is OCP MX
 *    v1.0's for E2M1. */
typedef struct mx_layer_opts {
  int activation;
  float alpha;
  float limit;
  int shared_expert;
  int act_fmt;
} mx_layer_opts;

/* moe_forward with layer options (see mx_layer_opts); the workspace size is
 * moe_workspace_size's.  Errors: as moe_forward, plus MX_ERR_INVALID_ARG for
 * an unknown option value or a non-positive / non-finite limit. */
MX_API int moe_forward_ex(const void* x_bf16, const float* logits, const void* w1_prep, const void* w2_prep,
                          int fmt, int T, int H, int I, int E, int k, float* out, void* ws, size_t ws_bytes,
                          const mx_layer_opts* opts, mx_stream_t stream);

/* moe_grouped_gemm_swiglu with layer options (the activation and act_fmt are
 * used: with MX_E2M1 the activation codes are MXFP4 [T, H/2] bytes and h is
 * written as MXFP4, [rows, I/2] bytes; shared_expert must be folded). */
MX_API int moe_grouped_gemm_swiglu_ex(const uint8_t* act_codes, const uint8_t* act_scales,
                                      const int32_t* offsets, const int32_t* sorted_slot, const void* w1_prep,
                                      int fmt, int T, int H, int I, int E, int k, uint8_t* h_codes,
                                      uint8_t* h_scales, void* ws, size_t ws_bytes, const mx_layer_opts* opts,
                                      mx_stream_t stream);

/* moe_grouped_gemm_down_combine with layer options: act_fmt MX_E2M1 reads
 * MXFP4 h ([rows, I/2] bytes; needs MXFP4 weights); the other fields must hold
 * their defaults' kind (the activation is not used here). */
MX_API int moe_grouped_gemm_down_combine_ex(const uint8_t* h_codes, const uint8_t* h_scales,
                                            const int32_t* offsets, const int32_t* sorted_slot,
                                            const float* topk_w, const void* w2_prep, int fmt, int T, int H,
                                            int I, int E, int k, float* out, void* ws, size_t ws_bytes,
                                            const mx_layer_opts* opts, mx_stream_t stream);

/* Kernel launches moe_forward_ex enqueues for this shape and these options
 * (host only; -1 for a rejected shape or option). */
MX_API int moe_forward_launches_ex(int T, int H, int I, int E, int k, int fmt, const mx_layer_opts* opts);

/* ---- the operators around the expert layer ---- */

/* element types of plain (unquantised) tensors */
#define MX_BF16 0
#define MX_F32 1

/* Residual addition, root-mean-square norm and MX quantisation in one pass:
 *   z = x + residual,  residual_out = z,
 *   y = z / sqrt(mean(z^2) + eps) * weight,  (codes, scales) = MX(y)
 * in fp32; residual_out, y and the codes are each rounded once from fp32 (the
 * codes by mx_quantize_act's rule, applied to the fp32 y: next to a rounding
 * border they may differ from the codes of the bf16 y).
 *   x [T, H] of x_type, residual [T, H] of residual_type or NULL (none),
 *   weight [H] of weight_type (each MX_BF16 or MX_F32).
 *   residual_out [T, H] of residual_type, given exactly where residual is; it
 *     may be residual itself, or x where the types are equal.
 *   y [T, H] bf16 or NULL.  codes [T, H] bytes (MX_E4M3) or [T, H/2]
 *     (MX_E2M1), scales [T, H/32]: both or neither.  y or codes is given.
 * Errors: MX_ERR_INVALID_ARG (null, T < 0, H <= 0, eps not positive and
 * finite, an unknown type or format), MX_ERR_UNSUPPORTED (H % 32, H > 32768),
 * MX_ERR_ALIGNMENT (a tensor other than scales not 16-byte aligned). */
MX_API int mx_add_rmsnorm(const void* x, int x_type, const void* residual, int residual_type, const void* weight,
                          int weight_type, int T, int H, float eps, void* residual_out, void* y, int fmt,
                          uint8_t* codes, uint8_t* scales, mx_stream_t stream);

/* Bytes of a weight [N, K] laid out for mx_linear (0 for sizes that it rejects). */
MX_API size_t mx_linear_prepared_bytes(int N, int K, int fmt);

/* Load-time layout of an MX weight for mx_linear, once for each weight.
 *   codes [N, K] (MX_E4M3) or [N, K/2] bytes (MX_E2M1), scales [N, K/32];
 *   dst: mx_linear_prepared_bytes bytes, 256-byte aligned.
 * Errors: MX_ERR_INVALID_ARG (null, sizes, format), MX_ERR_UNSUPPORTED (K % 32, K > 2^20,
 * N > 2^22), MX_ERR_ALIGNMENT (codes 16 bytes, dst 256), MX_ERR_WORKSPACE. */
MX_API int mx_linear_prepare(const uint8_t* codes, const uint8_t* scales, int N, int K, int fmt, void* dst,
                             size_t dst_bytes, mx_stream_t stream);

/* Bytes of workspace mx_linear needs for at most T tokens (0 for sizes that it rejects). */
MX_API size_t mx_linear_workspace_size(int T, int N, int K, int act_fmt);

/* A dense projection in MX:
 *   out[t, n] = bias[n] + sum_k A[t, k] * W[n, k]
 * with W the weight laid out by mx_linear_prepare and A the activations in act_fmt
 * (MX_E4M3, or with MX_E2M1 weights MX_E2M1): either x_bf16 [T, K], quantised within the
 * call as mx_quantize_act_ex does, or codes [T, K] (MX_E2M1: [T, K/2]) with scales
 * [T, K/32], as the norms and quantisers give them.  Products are exact, sums fp32, out
 * [T, N] (bf16 or fp32 by out_type) is rounded once.  bias [N] fp32 or NULL.
 * Deterministic.  ws: mx_linear_workspace_size bytes, its first word the status word.
 * Errors: MX_ERR_INVALID_ARG (null, sizes, an unknown format or type, both or neither of
 * x_bf16 and codes), MX_ERR_UNSUPPORTED (K % 32, K > 2^20, N or T > 2^22, MX_E2M1
 * activations with MX_E4M3 weights), MX_ERR_ALIGNMENT (x_bf16, codes, out 16 bytes,
 * w_prep, ws 256), MX_ERR_WORKSPACE, MX_ERR_CUDA. */
MX_API int mx_linear(const void* x_bf16, const uint8_t* codes, const uint8_t* scales, int act_fmt, const void* w_prep,
                     int w_fmt, const float* bias, int T, int N, int K, void* out, int out_type, void* ws,
                     size_t ws_bytes, mx_stream_t stream);

/* ---- gates of mx_sandwich_rmsnorm ---- */
#define MX_GATE_NONE 0
#define MX_GATE_CHANNEL 1 /* gate [H] */
#define MX_GATE_TOKEN 2   /* gate [T] */
#define MX_GATE_FULL 3    /* gate [T, H] */
#define MX_GATE_ACT_NONE 0
#define MX_GATE_ACT_SIGMOID 1

/* Norm behind a block, its gate and scale, the residual, and the norm ahead of the
 * next block with MX quantisation, in one pass:
 *   n = x / sqrt(mean(x^2) + eps) * post_weight   (n = x where post_weight is NULL)
 *   z = residual_scale * residual + block_scale * act(gate) * n,  residual_out = z,
 *   y = z / sqrt(mean(z^2) + eps) * weight,  (codes, scales) = MX(y)
 * in fp32; residual_out, y and the codes are each rounded once from fp32.
 *   x [T, H] of x_type, residual [T, H] of residual_type, post_weight and weight
 *     [H] (each MX_BF16 or MX_F32).
 *   gate: NULL with MX_GATE_NONE, else by gate_kind, of gate_type; act by gate_act.
 *   residual_out [T, H] of residual_type; it may be residual itself, or x where the
 *     types are equal.
 *   weight NULL: residual_out is the only output (y, codes and scales are NULL);
 *     else y [T, H] bf16 or NULL, codes and scales as mx_add_rmsnorm's, and y or
 *     codes is given.
 * Errors: MX_ERR_INVALID_ARG (null, T < 0, H <= 0, eps not positive and finite, a
 * scale that is not finite, an unknown type, gate or format), MX_ERR_UNSUPPORTED
 * (H % 32, H > 32768), MX_ERR_ALIGNMENT (a tensor other than scales and a token's
 * gate not 16-byte aligned). */
MX_API int mx_sandwich_rmsnorm(const void* x, int x_type, const void* post_weight, int post_weight_type,
                               const void* gate, int gate_type, int gate_kind, int gate_act, const void* residual,
                               int residual_type, float residual_scale, float block_scale, const void* weight,
                               int weight_type, int T, int H, float eps, void* residual_out, void* y, int fmt,
                               uint8_t* codes, uint8_t* scales, mx_stream_t stream);

/* A paged cache of keys and values in MX form.  Each of the four tables is
 * dense, [num_pages, n_kv_heads, page_size, row] with row = head_dim bytes of
 * codes (MX_E4M3; head_dim / 2 for MX_E2M1, element 2i in the low nibble) or
 * head_dim / 32 scale bytes: a page holds page_size tokens of one sequence,
 * head by head.  The tables are 16-byte aligned.  A scale byte of 255 is E8M0's
 * NaN: mx_kv_append never writes it, mx_kv_read gives NaN for its block, and the
 * attention a NaN row where a row sees such a key or value. */
typedef struct mx_kv_cache {
  uint8_t* k_codes;
  uint8_t* k_scales;
  uint8_t* v_codes;
  uint8_t* v_scales;
  int num_pages;
  int page_size;
  int n_kv_heads;
  int head_dim;
  int fmt; /* MX_E4M3 or MX_E2M1 */
} mx_kv_cache;

/* The three cache calls describe a batch in the same way, on the device:
 *   kv_lens [n_seqs]: tokens of each sequence in the cache, the new ones among
 *     them (they are its last);
 *   q_starts [n_seqs + 1]: new tokens q_starts[b] .. q_starts[b+1] - 1 of the
 *     [T, ...] tensors belong to sequence b (ascending from 0; a sequence may
 *     have none; rows from q_starts[n_seqs] on are padding);
 *   block_table [n_seqs, max_pages]: the page of each page_size tokens.
 * A length, start or page out of range sets MX_ERR_DEVICE_ARG in the workspace
 * status; nothing is read or written through it (see each call).  ws is a
 * 256-byte aligned, zero-filled workspace of at least 256 bytes, its first
 * word the status word. */

/* Quantises T new keys and values and writes them to their places in the cache:
 * token t of sequence b goes to position kv_lens[b] - q_starts[b+1] + t.
 *   k, v: bf16, token t's [n_kv_heads, head_dim] at t * stride elements.
 * The codes are mx_quantize_act's of the same row, bit for bit.  Skipped are the
 * tokens of a sequence whose start, end or length is out of range, and those
 * without a position (more new tokens than kv_lens counts) or a page.  Two
 * tokens with the same place leave either one.
 * Errors: MX_ERR_INVALID_ARG (null, negative or zero sizes, unknown format, a
 * stride below n_kv_heads * head_dim), MX_ERR_UNSUPPORTED (head_dim % 32),
 * MX_ERR_ALIGNMENT (k, v or a stride not a multiple of 16 bytes, a table),
 * MX_ERR_WORKSPACE. */
MX_API int mx_kv_append(const mx_kv_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                        const int32_t* block_table, const int32_t* kv_lens, const int32_t* q_starts, int n_seqs,
                        int max_pages, int T, void* ws, size_t ws_bytes, mx_stream_t stream);

/* ---- rotary positions ---- */
#define MX_ROPE_HALF 0        /* pairs (i, i + rot_dim / 2) */
#define MX_ROPE_INTERLEAVED 1 /* pairs (2i, 2i + 1) */
#define MX_ROPE_SCALING_NONE 0
#define MX_ROPE_SCALING_LINEAR 1
#define MX_ROPE_SCALING_NTK 2
#define MX_ROPE_SCALING_YARN 3
#define MX_ROPE_SCALING_BANDS 4

/* The table that mx_rope_kv_append rotates by (host only: plain memory, no GPU).
 * Pair i of rot_dim / 2 turns by f_i = base^(-2i / rot_dim) radians a position:
 *   turns[i] = the fraction of f_i / 2 pi, in units of 2^-64; *amplitude = 1;
 * scaled for contexts `factor` times as long as the original_length:
 *   NONE    as it is (factor, low, high and original_length are not used)
 *   LINEAR  f_i / factor
 *   NTK     base * factor^(rot_dim / (rot_dim - 2)) in the place of base
 *   YARN    with d(t) = rot_dim ln(original_length / (2 pi t)) / (2 ln base), the pair
 *           that turns t times in the original length: f_i for i up to floor(d(high)),
 *           f_i / factor from ceil(d(low)) on, a linear ramp between them (the two
 *           held to [0, rot_dim - 1]); *amplitude = 0.1 ln(factor) + 1
 *   BANDS   by t_i, pair i's turns in the original length: f_i for t_i >= high,
 *           f_i / factor for t_i <= low, and s f_i + (1 - s) f_i / factor with
 *           s = (t_i - low) / (high - low) between them
 * (YARN after "YaRN: Efficient Context Window Extension of Large Language Models".)
 * Errors: MX_ERR_INVALID_ARG (null, rot_dim not positive and even, an unknown
 * scaling; base <= 1, and where they are used factor < 1, original_length <= 0, not
 * 0 < low < high, or not finite; NTK with rot_dim 2). */
MX_API int mx_rope_table(int rot_dim, double base, int scaling, double factor, double low, double high,
                         int original_length, uint64_t* turns, float* amplitude);

/* mx_kv_append with rotary positions: of each token that mx_kv_append would write,
 * the first rot_dim elements of every head of q and k are rotated,
 *   (a, b) -> amplitude * (a cos t - b sin t, a sin t + b cos t),  t = position * f_i,
 * the others pass; the rotated k (from its fp32 values: one rounding) and v go to their
 * places in the cache, the rotated q goes to q_out as bf16.
 *   q: bf16, token t's [n_q_heads, head_dim] at t * q_stride elements, or NULL with
 *     n_q_heads 0 (then no q_out).  q_out the same at t * q_out_stride; it may be q
 *     with the same stride, and else does not overlap q, k or v.
 *   positions [T] int32 or NULL: the angles' positions; without them a token's place in
 *     its sequence.  They do not move the place that is written.
 *   turns [rot_dim / 2] on the device, amplitude: mx_rope_table's.  An angle is exact to
 *     2^-32 turns for the table's frequencies, which are f_i in 64-bit arithmetic: another
 *     2^-52 turns a position (2^-32 at position 2^20), more for BANDS with low next to high.
 * Tokens that are skipped leave their rows of q_out as they were.
 * Errors: as mx_kv_append (with q, q_out and their strides), plus MX_ERR_INVALID_ARG (an
 * unknown layout, rot_dim < 0 or > head_dim, amplitude not finite, q without q_out) and
 * MX_ERR_UNSUPPORTED (rot_dim % 16, head_dim > 256, n_q_heads * head_dim > 2^20). */
MX_API int mx_rope_kv_append(const mx_kv_cache* cache, const void* q, int64_t q_stride, int n_q_heads, void* q_out,
                             int64_t q_out_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const int32_t* positions, const uint64_t* turns, int rot_dim, int layout,
                             float amplitude, const int32_t* block_table, const int32_t* kv_lens,
                             const int32_t* q_starts, int n_seqs, int max_pages, int T, void* ws, size_t ws_bytes,
                             mx_stream_t stream);

/* The reverse: the last q_starts[b+1] - q_starts[b] tokens of each sequence
 * (all of them where q_starts counts kv_lens) as bf16 [T, n_kv_heads, head_dim],
 * dense.  A code's value times its scale is exact in bf16 (but for overflow
 * and bf16's subnormals, rounded to nearest even).  Rows of padding and of bad
 * lengths, starts or pages are zero.  Errors as mx_kv_append. */
MX_API int mx_kv_read(const mx_kv_cache* cache, const int32_t* block_table, const int32_t* kv_lens,
                      const int32_t* q_starts, int n_seqs, int max_pages, int T, void* k_out, void* v_out, void* ws,
                      size_t ws_bytes, mx_stream_t stream);

/* Bytes of workspace mx_paged_attention needs for at most T tokens, n_seqs
 * sequences and max_q_len new tokens in one of them (0 for a shape that it
 * rejects). */
MX_API size_t mx_paged_attention_workspace_size(int T, int n_seqs, int n_heads, int n_kv_heads, int head_dim,
                                                int max_q_len);

/* Attention of new tokens over the cache (which holds their keys and values
 * already): for new token i of n of a sequence with kv keys, and query head h,
 *   s_j = scale * q . k_j,  o = sum_j softmax(s)_j v_j,  lse = log sum_j exp s_j
 * over its visible keys j: j < kv; with causal != 0, j <= kv - n + i; with
 * window > 0 (causal only), also j > kv - n + i - window.  A row with no
 * visible key gets o = 0 and lse = -inf.
 *   q: bf16, token t's [n_heads, head_dim] at t * q_stride elements; query
 *     heads h * (n_heads / n_kv_heads) .. share KV head h.
 *   out [T, n_heads, head_dim] bf16, lse [T, n_heads] fp32 or NULL, dense.
 *   max_q_len: no sequence has more new tokens (one that has is reported and
 *     its rows are not written).
 * Scores, softmax statistics and sums are fp32.  For the second product a weight
 * is rounded to f16 (2^-11), or, in chunks where the V scales of 64 keys spread over
 * more than 2^15, to bf16 (2^-8); a weight times its value's largest block scale is
 * held to 2^-25 of the row's largest such product: next to a value 2^25 larger, the
 * others fade.  For few rows an element of a key or value is held to 2^-25 of its
 * token's largest block scale, and is zero where its own block's scale lies 2^25
 * below (MX_E2M1: 2^31).
 * Rows of padding and of bad metadata are not written; a bad page's keys are left
 * out.  Starts that are not ascending and ask for more work than the sizes allow are
 * reported, and no row is written.  Cache places that no row sees may hold anything, also pages behind the
 * window may be gone.
 * A NaN or infinity in a query makes its row NaN; a NaN among the values that
 * some new token sees may reach the sequence's other new tokens of the call.
 * Deterministic: the same call gives the same bits.  One kernel for few rows, one
 * for chunks, or both in two launches: the choice goes by the sizes, among them how
 * many keys a sequence may have by max_pages * page_size and the window, so a block
 * table should be no wider than the batch needs.
 * Errors: MX_ERR_INVALID_ARG (null, sizes, n_heads % n_kv_heads, scale or
 * scale * log2(e) not positive and finite, window < 0 or without causal, stride),
 * MX_ERR_UNSUPPORTED (head_dim other than 64 and 128, page_size % 16, more
 * than 2^30 rows of q or 2^31 of a cache table, or 2^31 (256 query rows x 64
 * keys) of work for one KV head, 4e9 in all, by the sizes given),
 * MX_ERR_ALIGNMENT, MX_ERR_WORKSPACE, MX_ERR_CUDA. */
MX_API int mx_paged_attention(const mx_kv_cache* cache, const void* q, int64_t q_stride, int n_heads,
                              const int32_t* block_table, const int32_t* kv_lens, const int32_t* q_starts, int n_seqs,
                              int max_pages, int T, int max_q_len, float scale, int causal, int window, void* out,
                              float* lse, void* ws, size_t ws_bytes, mx_stream_t stream);

/* Bytes of workspace mx_sample needs (0 for sizes that it rejects). */
MX_API size_t mx_sample_workspace_size(int T, int V);

/* One token for each row of logits, drawn by a given random number.  With the row's
 * tokens in the order of their logits (descending; the same logit: ascending number):
 *   weights  w_i = exp((logit_i - max) / temperature)
 *   top_k    the first top_k tokens are kept (top_k <= 0 or >= V: all)
 *   top_p    of those, token i is kept while the weight of those before it is below
 *            top_p times the weight of all those (top_p >= 1: all; the first always)
 *   min_p    of those, the ones with w_i >= min_p (of the largest; above 1 counts as 1)
 *   token    the first, by number, at which the sum of the kept weights exceeds u
 *            times their whole sum; logp = log of its weight's share in that sum.
 * temperature 0 or top_k 1: the largest logit (of the lowest number), logp 0; other
 * temperatures are held to [2^-126, 2^100].
 *   logits [T, V] bf16 or fp32 (type), row t at t * stride elements.
 *   temperature, top_p, min_p fp32, top_k int32: [T] each, or NULL for 1, 1, 0, 0.
 *   u [T] fp32 in [0, 1) (held to it, a NaN counts as 0).  tokens [T] int32, logp [T] fp32 or NULL.
 * Weights are held as whole multiples of 2^-43 (those below 2^-44 are never drawn), 2^-30 off
 * (those of bf16 logits below 2^-16 of the largest 2^-22), and summed exactly: the same call
 * gives the same tokens, and one next to a border may differ from exact arithmetic.  In logp a
 * logit's distance from the maximum is in fp32.  Logits of -inf are never drawn; of +inf, the
 * only ones drawn.  A row with a NaN, without a finite or infinite maximum, with a negative
 * temperature or a NaN among its rules gives token -1 and logp NaN and sets
 * MX_ERR_DEVICE_ARG in the workspace status.
 * Errors: MX_ERR_INVALID_ARG (null, T < 0, V <= 0, an unknown type, stride < V),
 * MX_ERR_UNSUPPORTED (V > 800000 in bf16, V > 400000 in fp32, T >= 2^27), MX_ERR_ALIGNMENT (a tensor
 * not aligned to its elements, ws), MX_ERR_WORKSPACE, MX_ERR_CUDA. */
MX_API int mx_sample(const void* logits, int type, int64_t stride, int T, int V, const float* temperature,
                     const int32_t* top_k, const float* top_p, const float* min_p, const float* u, int32_t* tokens,
                     float* logp, void* ws, size_t ws_bytes, mx_stream_t stream);

/* Copy the workspace status word to *host_status (synchronising `stream`) and
 * clear it.  0 = no device-side error; otherwise an MX_ERR_* code. */
MX_API int moe_get_status(void* ws, mx_stream_t stream, int* host_status);

/* *id = a number of the graph capture that `stream` is part of, 0 where it is part of none:
 * for callers that keep a workspace for each graph.  (Two graphs that may run at once need
 * one each, and a zero fill that was captured into one graph is none for the other.)
 * Errors: MX_ERR_INVALID_ARG (null), MX_ERR_CUDA. */
MX_API int mx_capture_id(mx_stream_t stream, uint64_t* id);

/* Exchanges *mode with the calling thread's capture mode, as cudaThreadExchangeStreamCaptureMode
 * does: 0 global, 1 this thread, 2 relaxed.  A thread that captures one stream into a graph may
 * allocate, fill and wait for memory on another while its mode is relaxed.
 * Errors: MX_ERR_INVALID_ARG (null, another mode), MX_ERR_CUDA. */
MX_API int mx_exchange_capture_mode(int* mode);

/* Test hook: the wall-clock limit, in nanoseconds, of every bounded wait inside
 * the GEMM kernels (default 2e9).  A tiny limit makes the waits run out, which
 * exercises the MX_ERR_TIMEOUT path without hanging the GPU. */
MX_API void mx_debug_set_wait_limit_ns(uint64_t ns);

/* Measurement hook: while enabled (enable != 0), each grouped-GEMM kernel
 * launch is bracketed by two CUDA events the library records on the launch's
 * stream (the first 4096 launches after enabling; events of the device that is
 * current at the first recorded launch, later launches on another device are
 * not recorded).  mx_debug_gemm_times waits for the recorded events, writes for
 * the first min(n, max) launches the kernel's device time in milliseconds
 * (ms[i]) and its epilogue (epi[i]: 0 gate/up, 1 down), forgets them and
 * returns n, the number recorded (-1: a CUDA error).  Enabling or disabling
 * also forgets them.  Not for streams being captured into a CUDA graph.  The
 * pages have no counterpart: it times the dominant kernel apart from the row
 * gather that shares its call. */
MX_API void mx_debug_time_gemms(int enable);
MX_API int mx_debug_gemm_times(float* ms, int* epi, int max);

/* Hash of the sources, flags and compiler this library was built from
 * (16 hex digits; static string).  Lets a caller check that the library it
 * loaded was compiled from the sources it expects. */
MX_API const char* mx_build_stamp(void);

#ifdef __cplusplus
}
#endif
#endif /* MXMOE_H_ */
