/*
 * moe_w4.h -- C ABI of the GB300 (sm_103a) W4A16 mixture-of-experts block.
 *
 * The block is the expert layer of a Qwen3.6-35B-A3B-style model as described
 * in "Perplexity libera Lily, un motor de IA que supera a MLX-LM en Apple
 * Silicon" (diariobitcoin.com):
 *   - section "Qwen3.6 combina tres cargas de trabajo": a router scores all E
 *     (256) experts and selects k (8) per token; one shared expert processes
 *     every token; weights are 4-bit affine with groups of 64, one bfloat16
 *     scale and one bfloat16 bias per group;
 *   - section "Las optimizaciones en el prefill": the grouped GEMM rebuilds
 *     weights block by block on chip and accumulates in FP32 (the dequantised
 *     array never exists in memory), and the routing histogram, prefix scan,
 *     scatter and block map stay on the GPU with no CPU synchronisation
 *     inside a layer.
 *
 * Conventions for every call:
 *   - All tensor arguments are DEVICE pointers owned by the caller, on the
 *     plan's device, 16-byte aligned. bf16 tensors are passed as uint16_t bit
 *     patterns. The library never frees or keeps caller memory past a call.
 *   - A plan owns only its device scratch, allocated once in moe_plan_create
 *     and sized for max_tokens.
 *   - Calls are stream-ordered and asynchronous: they enqueue kernels on
 *     `stream` (NULL = legacy default stream) and never wait for the device.
 *     Grid sizes never depend on routing results, so no value is read back.
 *   - Argument errors are found on the host before any launch and returned as
 *     a status; nothing is enqueued then. Errors found on the device (a
 *     bounded wait that ran out) are latched in a device word and reported by
 *     moe_get_error.
 *   - Weights (router weights, packed experts, scales, biases) are read by
 *     some kernels before they wait for the previous launch on the stream
 *     (programmatic dependent launch): no kernel running just before a call
 *     on the same stream may write them (record an event, or run any other
 *     launch in between). Token inputs are always read after that wait.
 *   - A plan is not thread-safe: calls on one plan must come from one host
 *     thread at a time, and calls that share a plan's scratch must be ordered
 *     on the device (same stream, or explicit events).
 *   - Operand precision. The pages fix only FP32 accumulation and the bf16
 *     scale and bias. The expert GEMMs multiply fp16 operands: token values
 *     are converted from bf16 to fp16 (exact for magnitudes up to 65504;
 *     below 2^-14 they become fp16 subnormals, an absolute error under
 *     2^-25, negligible against a unit-scale row), the tensor-core path
 *     rebuilds each weight as fp16(q * scale + bias) from fp16 copies of the
 *     scale and bias, and the SwiGLU activations are stored as fp16. The
 *     contract, checked on the device:
 *       |x| < 65536 for every token value (a larger one, an inf or a NaN is
 *         clamped to +-65504 and flagged), checked on every call;
 *       every scale is 0 or has magnitude in [2^-14, 2^12) and every bias
 *         has magnitude below 2^11 (then |q * scale + bias| < 65504 and no
 *         scale is an fp16 subnormal), checked once per weight set, by a
 *         kernel on the stream the first time a plan sees the set (by its
 *         scale and bias addresses; new values written in place at the
 *         same addresses are not checked again).
 *     A value outside the contract sets a bit in the plan's device error
 *     word that moe_get_error reports as MOE_ERR_OPERAND_RANGE; the call
 *     itself still completes with clamped values. The activations the
 *     block produces itself (RMS-normalised stack input, SwiGLU outputs of
 *     in-contract weights) stay far inside these bounds.
 */
#ifndef MOE_W4_H
#define MOE_W4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t compatible handle, so this header needs no CUDA headers */
typedef struct CUstream_st* moe_stream_t;

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,    /* null/misaligned pointer, bad size, bad field */
  MOE_ERR_UNSUPPORTED = 2,    /* valid request this build has no kernel for */
  MOE_ERR_CUDA = 3,           /* a CUDA runtime/driver call failed */
  MOE_ERR_CAPACITY = 4,       /* T above the plan's max_tokens */
  MOE_ERR_DEVICE_TIMEOUT = 5, /* a device-side bounded wait ran out */
  MOE_ERR_OPERAND_RANGE = 6   /* an input outside the fp16 operand range (below) */
} moe_status;

/* Plan description. Sizes are in elements. */
typedef struct {
  int hidden;            /* H: model width (2048); multiple of group_size */
  int inter;             /* I: expert FFN width (512); multiple of group_size */
  int num_experts;       /* E: routed experts (256); 8..512, multiple of 8 */
  int top_k;             /* k: experts per token (8); 1..min(E, 32) */
  int group_size;        /* G: quantisation group along K; must be 64 */
  int has_shared;        /* 1: one always-on shared expert with weight 1 */
  int max_tokens;        /* capacity: scratch is sized for this T, once */
  int block_m;           /* rows per block-map tile; must be 128 */
  int gemm_path;         /* 0 auto, 1 tensor-core (tcgen05) path, 2 small-M path,
                            3 tensor-core path on SM pairs (tcgen05 cta_group::2;
                            falls back to 1 on a device without cluster launch) */
  int small_m_max_tokens;/* auto: T <= this uses the small-M path (default 16 if 0) */
  int wait_limit_ms;     /* device bounded-wait limit (default 1000 if 0) */
} moe_plan_desc;

typedef struct moe_plan* moe_plan_t;

/* One 4-bit affine matrix set for E experts, N output rows, K inputs.
 * Weight W[e][n][kk] = q * scale[e][n][kk/64] + bias[e][n][kk/64] where q is
 * nibble (kk % 8) -- bits 4*(kk%8) .. 4*(kk%8)+3 -- of qweight[e][n][kk/8],
 * read as an unsigned integer 0..15. */
typedef struct {
  const uint32_t* qweight;   /* [E][N][K/8] */
  const uint16_t* scales;    /* [E][N][K/64] bf16 */
  const uint16_t* biases;    /* [E][N][K/64] bf16 */
} moe_w4;

/* SwiGLU expert set: gate and up are N = inter, K = hidden; down is
 * N = hidden, K = inter. An expert computes
 *   a[n] = silu(sum_k x[k] Wg[n][k]) * sum_k x[k] Wu[n][k],
 *   out[m] = sum_n a[n] Wd[m][n]. */
typedef struct {
  moe_w4 gate, up, down;
} moe_experts;

/* Routing result. moe_route fills this with pointers into plan scratch that
 * stay valid until the next moe_route / moe_forward_layer on the plan. A
 * caller may also point it at its own device buffers with these layouts
 * (slot s = t*k + j, position = row in expert-contiguous order):
 *   topk_idx     int32 [T][k]  selected experts, rank order (logit desc,
 *                              lower index first on ties)
 *   topk_w       f32   [T][k]  softmax over all E, renormalised over the k
 *   counts       int32 [E]     histogram of selected experts
 *   offsets      int32 [E+1]   exclusive prefix scan of counts; [E] = T*k
 *   tile_offsets int32 [E+1]   exclusive scan of ceil(counts/block_m)
 *   perm         int32 [T*k]   position -> slot, stable in token order
 *   inv          int32 [T*k]   slot -> position
 *   block_map    int32 [tiles][3] (expert, first position, rows) per tile,
 *                              expert-major; shared-expert tiles excluded
 *   num_tiles    int32 [1]     number of block_map tiles
 *   logits       f32   [T][E]  router logits (moe_route only; may be NULL
 *                              when the struct is given to
 *                              moe_grouped_w4_ffn) */
typedef struct {
  int32_t* topk_idx;
  float* topk_w;
  int32_t* counts;
  int32_t* offsets;
  int32_t* tile_offsets;
  int32_t* perm;
  int32_t* inv;
  int32_t* block_map;
  int32_t* num_tiles;
  float* logits;
} moe_routing;

/* Create a plan on CUDA device `device`: validates `desc` (host only; no
 * CUDA call is made when it is invalid) and allocates the scratch. */
moe_status moe_plan_create(const moe_plan_desc* desc, int device, moe_plan_t* out);

/* Free the plan and its scratch. Waits for the device to finish using it. */
moe_status moe_plan_destroy(moe_plan_t plan);

/* Bytes of device scratch a plan with this description allocates (host only). */
moe_status moe_plan_scratch_bytes(const moe_plan_desc* desc, size_t* bytes);

/* Routing (histogram, prefix scan, scatter and block map in section "Las
 * optimizaciones en el prefill"; router and top-8 in section "Qwen3.6
 * combina tres cargas de trabajo"):
 *   logits[t][e] = sum_h x[t][h] * router_w[h][e] + router_bias[e]  (FP32)
 * then top-k, weights, counts, offsets, tile offsets, perm, inv, block map.
 * x: bf16 [T][H]; router_w: bf16 [H][E]; router_bias: f32 [E] or NULL.
 * `out` receives pointers into plan scratch. 1 <= T <= max_tokens. */
moe_status moe_route(moe_plan_t plan, const uint16_t* x, int T, const uint16_t* router_w,
                     const float* router_bias, moe_routing* out, moe_stream_t stream);

/* Experts on a given routing (the grouped GEMM with block-wise dequant in
 * section "Las optimizaciones en el prefill"):
 *   y[t] = shared(x[t]) + sum_j topk_w[t][j] * expert_{topk_idx[t][j]}(x[t])
 * x: bf16 [T][H]; routing: as moe_route produces (topk_w, perm, inv,
 * block_map and num_tiles are read); routed: E experts; shared: one expert
 * set with E = 1, or NULL (must be non-NULL iff desc.has_shared);
 * y: f32 [T][H], the block's FP32 sum (the pages accumulate in FP32; a bf16
 * rounding of y alone would cost about 1.5% of the output's rms at 4-sigma
 * values), must not overlap x. Dequantised weights exist only in on-chip
 * memory. Routed experts' outputs are weighted and kept in bf16 before the
 * combine; the shared expert's are kept in FP32. */
moe_status moe_grouped_w4_ffn(moe_plan_t plan, const uint16_t* x, int T,
                              const moe_routing* routing, const moe_experts* routed,
                              const moe_experts* shared, float* y, moe_stream_t stream);

/* moe_route followed by moe_grouped_w4_ffn: one MoE layer, no host sync. */
moe_status moe_forward_layer(moe_plan_t plan, const uint16_t* x, int T,
                             const uint16_t* router_w, const float* router_bias,
                             const moe_experts* routed, const moe_experts* shared,
                             float* y, moe_stream_t stream);

/* moe_forward_layer followed by moe_residual_add(x, y, T, alpha, x, xn_out)
 * in one call whose last pass updates the stack directly from the experts'
 * outputs, so y is never written (the FP32 [T][H] round trip is saved):
 *   y = moe(xn); x = bf16(x + alpha * y); xn_out = bf16(rmsnorm(x))
 * Bit-identical to the two calls. xn (the layer's input) and xn_out may be
 * the same buffer (the update runs after every read of xn); x must differ
 * from both. Layouts as in moe_forward_layer and moe_residual_add. */
moe_status moe_forward_layer_residual(moe_plan_t plan, const uint16_t* xn, int T,
                                      const uint16_t* router_w, const float* router_bias,
                                      const moe_experts* routed, const moe_experts* shared,
                                      float alpha, uint16_t* x, uint16_t* xn_out,
                                      moe_stream_t stream);

/* One layer of a stack for moe_forward_stack: its router and experts.
 * shared is ignored (may be NULL) when the plan has no shared expert. */
typedef struct {
  const uint16_t* router_w;     /* bf16 [H][E] */
  const float* router_bias;     /* f32 [E] or NULL */
  moe_experts routed;
  moe_experts shared;
} moe_layer;

/* A stack of MoE layers on a prompt of any length (chunked prefill; the
 * pages' engine prefills long prompts in chunks, "Las optimizaciones en el
 * prefill"). x is the residual stream, bf16 [T][H], updated in place:
 *   xn = bf16(rmsnorm(x));
 *   for each layer: x = bf16(x + alpha * moe_layer(xn)); xn = bf16(rmsnorm(x))
 * T may exceed the plan's max_tokens: the tokens go through all layers in
 * chunks of at most max_tokens rows, one chunk after the other (the block
 * treats every token on its own, so each chunk's result is the one of the
 * whole prompt). xn is caller scratch, bf16 [min(T, max_tokens)][H], and holds
 * the last chunk's normalised stream on return. Every layer of a chunk is one
 * moe_forward_layer_residual, except for decode-sized chunks (at most 8
 * tokens, on the small-M path): there every layer is one launch of a fused
 * kernel that takes the RMS norm, routes, runs both expert passes and
 * updates x (the same arithmetic up to rounding: the routed experts' outputs
 * stay FP32 until the combine; the routing lands in the plan's routing
 * arrays and y in its FP32 shared-output buffer, moe_debug_buffer 3).
 * Stream-ordered, no host sync. Errors: as for the per-layer calls (checked
 * for every layer before any launch); MOE_ERR_INVALID_ARG for num_layers < 1
 * or a NULL layers array. */
moe_status moe_forward_stack(moe_plan_t plan, uint16_t* x, uint16_t* xn, int T,
                             const moe_layer* layers, int num_layers, float alpha,
                             moe_stream_t stream);

/* Update between stacked layers (not part of the expert block itself):
 *   x_out[t] = bf16(x[t] + alpha * y[t])                 (skipped if y == NULL)
 *   xn_out[t] = bf16(x_out[t] / sqrt(mean_h x_out[t][h]^2 + 1e-6))
 *                                                        (skipped if NULL)
 * x, x_out, xn_out bf16 [T][H]; y f32 [T][H]; FP32 arithmetic, the mean of
 * squares over the bf16-rounded x_out. x_out may equal x (NULL means x);
 * xn_out must be a separate buffer. xn_out is the RMS-normalised input of
 * the next layer: without it the SwiGLU experts, quadratic in their input,
 * make a residual stack grow without bound. */
moe_status moe_residual_add(moe_plan_t plan, const uint16_t* x, const float* y, int T,
                            float alpha, uint16_t* x_out, uint16_t* xn_out,
                            moe_stream_t stream);

/* Routing without a plan and without any device allocation. The pages have
 * no counterpart: this entry point exists for callers that cannot call
 * cudaMalloc -- a host framework that hands out all device memory from its
 * own pool (an allocation behind its back can fail or fragment the memory
 * it budgets), runtimes with no device allocator at all, and latency-bound
 * callbacks that must not block (cudaMalloc can synchronise the device).
 * It computes exactly what moe_route computes, with the same kernels.
 * The caller passes x, router_w, router_bias (may be NULL) as for moe_route
 * and every output buffer in `out` (layouts as in moe_routing; block_map
 * must hold ceil(T*k/128) + E triples; logits is required, every buffer
 * 8-byte aligned; hidden a multiple of 64, num_experts a multiple of 8 and
 * at least 8, 1 <= top_k <= num_experts, otherwise MOE_ERR_INVALID_ARG;
 * top_k above 32 returns MOE_ERR_UNSUPPORTED as for a plan). Every input is
 * read only after the previous work on the stream has completed, so the
 * caller's own kernel just before may write x or the router weight.
 * The library's only scratch for this call is a fixed device array of
 * 128 x 512 int32 (256 KB) in the library image, present on every GPU that
 * loads the library until the process exits; hence T <= 4096 and
 * num_experts <= 512, and larger requests return MOE_ERR_CAPACITY. Nothing
 * in that array needs clearing between calls. The first call on a device
 * looks up the array's device address (a host-side runtime query, with that
 * device current) and keeps it for later calls. All calls share the array:
 * calls that can overlap on the GPU (different streams without ordering)
 * race and must not be made.
 * A bounded wait of the routing kernels that runs out (1 s) leaves the
 * outputs unspecified and is reported by moe_route_noalloc_get_error. */
moe_status moe_route_noalloc(const uint16_t* x, int T, int hidden, const uint16_t* router_w,
                             const float* router_bias, int num_experts, int top_k,
                             const moe_routing* out, moe_stream_t stream);

/* Reads and clears the device error word of moe_route_noalloc on the
 * current device (shared by every call on that device). Synchronises the
 * device: call it between steps, never inside one. Returns MOE_OK,
 * MOE_ERR_DEVICE_TIMEOUT, or MOE_ERR_CUDA if the context has failed. Not
 * part of the pages' method: the error path of the call above. */
moe_status moe_route_noalloc_get_error(void);

/* Launches, on `stream`, a kernel whose bounded wait can never be satisfied,
 * with the given limit (1 us .. 10 s) and the error word of
 * moe_route_noalloc: it gives up, latches MOE_ERR_DEVICE_TIMEOUT there and
 * exits, so a test can check moe_route_noalloc_get_error without faulting
 * or hanging the GPU. */
moe_status moe_route_noalloc_debug_wait_timeout(int limit_us, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * Operators of the layer around the expert block. The pages describe only the
 * block; these are its neighbours in a served pre-norm layer: the residual's
 * addition and RMS norm before it, a router's choice by scores, bias and
 * groups, and 4-bit projections that carry the low-rank adapters of many
 * requests at once.
 * ------------------------------------------------------------------------- */

/* Residual addition, RMS norm and 8-bit output. */
typedef struct {
  int hidden;              /* H: columns of a row; a multiple of 8, 8..16384 */
  float eps;               /* added to the mean of squares; >= 0, finite */
  float alpha;             /* factor of delta; finite */
  int delta_f32;           /* delta's type: 0 bf16, 1 f32 (an expert block's y) */
  int quant_group;         /* columns per 8-bit scale: 0 the whole row, or 128 */
  long long x_stride;      /* elements between rows of x and of x_out; 0 = H */
  long long delta_stride;  /* of delta; 0 = H */
  long long out_stride;    /* of xn_out and of q_out; 0 = H */
} moe_norm_desc;

/* For every row t of T:
 *   x_out = bf16(x + alpha * delta)              (x when delta is NULL)
 *   v     = x_out / sqrt(mean_h x_out^2 + eps) * weight   (weight NULL: 1)
 *   xn_out = bf16(v)
 *   q_scale = max|v| / 448 over the row or over each 128 columns (the last
 *             group of a row may be shorter)
 *   q_out   = e4m3(v * 448 / max|v|), round to nearest even
 * FP32 arithmetic; the mean of squares is over the bf16-rounded x_out, and v
 * is quantised from its FP32 value, not from xn_out. A group whose max|v| is
 * below 2^-100 gets scale 0 and codes 0. A NaN in a row makes its outputs and
 * scales NaN.
 * x bf16, delta bf16 or f32, weight bf16 [H] or NULL; x_out and xn_out bf16,
 * q_out e4m3 bytes, q_scale f32 [T][1 or ceil(H/128)]. Each output may be
 * NULL, but not all; q_out and q_scale come together. x_out may equal x (with
 * the same rows); no other output may overlap an input or another output, each
 * taken from its first row to the end of its last, with what a stride leaves out.
 * Pointers 16-byte aligned, strides multiples of 8 and at least H. Needs no
 * plan; runs on the current device. T >= 1. */
moe_status moe_norm_quant(const moe_norm_desc* desc, const uint16_t* x, const void* delta,
                          const uint16_t* weight, int T, uint16_t* x_out, uint16_t* xn_out,
                          uint8_t* q_out, float* q_scale, moe_stream_t stream);

/* How moe_route_scored scores and chooses. */
typedef struct {
  int score;               /* p = 0: softmax over all E, 1: sigmoid of the logit */
  int groups;              /* the E experts in this many equal runs; 1..32, divides E */
  int topk_groups;         /* groups a token may choose from; 1..groups */
  int renormalise;         /* 1: the k weights are divided by their sum */
  float scale;             /* factor of the weights, last; finite */
  const float* bias;       /* f32 [E] added to p for the choice only, or NULL */
} moe_score_desc;

/* Router logits alone (the first step of moe_route, the same bits):
 *   logits[t][e] = sum_h x[t][h] * router_w[h][e] + router_bias[e]
 * logits: f32 [T][E], 16-byte aligned, caller's. Other arguments as moe_route. */
moe_status moe_router_logits(moe_plan_t plan, const uint16_t* x, int T, const uint16_t* router_w,
                             const float* router_bias, float* logits, moe_stream_t stream);

/* Routing by scores, from given logits f32 [T][E]:
 *   p = softmax or sigmoid of the logits; c = p + bias (no bias: the logits'
 *   own order); with groups, a group's score is the sum of its two largest c
 *   (p without a bias; its one c in groups of one), and only the topk_groups
 *   best groups' experts are eligible; the k largest c of those are chosen, in
 *   descending order; weight = p, over the chosen ones' sum if renormalise,
 *   times scale.
 * Equal values go to the lower index, of experts and of groups. The choice is
 * that of 64-bit scores: where 32-bit ones lie too close to tell, they are
 * taken again in 64 bits. A NaN logit counts as -infinity; a row with no
 * finite maximum has p = 0 under softmax. An expert whose bias is -infinity
 * or NaN is closed: chosen only when nothing else is eligible, and then with
 * weight 0. Weights whose sum is 0 stay 0.
 * Then counts, offsets, tile offsets, perm, inv and block map as moe_route
 * makes them. `routing`: every field that is NULL receives the plan's scratch
 * pointer; the others are the caller's device buffers (layouts of
 * moe_routing, 4-byte aligned; block_map holds ceil(T*k/128) + E triples, of
 * which num_tiles are written); `logits` is ignored. The result can be given
 * to moe_grouped_w4_ffn. Errors: MOE_ERR_INVALID_ARG also when the eligible
 * groups hold fewer than k experts. */
moe_status moe_route_scored(moe_plan_t plan, const float* logits, int T,
                            const moe_score_desc* desc, moe_routing* routing,
                            moe_stream_t stream);

/* A 4-bit projection with adapters: its sizes. */
typedef struct {
  int in_features;         /* K: a multiple of 64, at most 16384 */
  int out_features;        /* N: 1..1048576 */
  int max_tokens;          /* capacity: scratch is sized for this T, once */
  int max_rank;            /* largest adapter rank: a multiple of 8, 0..128; 0: none */
  int wait_limit_ms;       /* device bounded-wait limit (default 1000 if 0) */
} moe_linear_desc;

typedef struct moe_linear* moe_linear_t;

/* n low-rank adapters of one rank r on a K -> N projection. */
typedef struct {
  const uint16_t* a;       /* bf16 [n][r][K] */
  const uint16_t* b;       /* bf16 [n][N][r] */
  const float* scale;      /* f32 [n], or NULL: 1 */
  int n;                   /* adapters, 1..65536 */
  int rank;                /* r: a multiple of 8, 8..max_rank */
} moe_lora;

typedef enum { MOE_X_BF16 = 0, MOE_X_E4M3 = 1 } moe_x_type;

moe_status moe_linear_create(const moe_linear_desc* desc, int device, moe_linear_t* out);
moe_status moe_linear_destroy(moe_linear_t linear);
moe_status moe_linear_scratch_bytes(const moe_linear_desc* desc, size_t* bytes);

/* For every row t of T, with W as in moe_w4 (E = 1) and a = adapter[t]:
 *   y[t] = bf16(x_scale[t] * (x[t] W^T + scale[a] * (x[t] A[a]^T) B[a]^T))
 * adapter: int32 [T]; a value outside 0..n-1 (such as -1) means no adapter.
 * lora and adapter are both NULL or both given. x: bf16 with x_scale NULL, or
 * e4m3 bytes with x_scale f32 [T] (moe_norm_quant's row scales) or NULL (1).
 * x_stride and y_stride: elements between rows, 0 = K and N; x_stride is a
 * multiple of 16, y_stride at least N. x, x_scale and the weights 16-byte
 * aligned, y and adapter 4-byte. y overlaps no input, each taken from its first
 * row to the end of its last. Rows may come in any
 * order of adapters; rows of one adapter next to each other are fastest.
 * The sums are FP32; weights are rebuilt as fp16(q * scale + bias) and bf16
 * rows enter as fp16 under the operand contract above, reported by
 * moe_linear_get_error; x A^T is kept to 16 significant bits. A token's row
 * depends on its own x, scale and adapter alone: infinities and NaNs of another
 * token or another adapter do not reach it. An infinity or NaN in an adapter's
 * own arrays shows in its tokens' outputs that it feeds, as an infinity, a NaN or
 * a value of the size of the largest bf16 times x A^T. Weights and adapters (a, b, scale) are read
 * under the rule for weights above; x, x_scale and the ids in `adapter` only
 * once every earlier launch on the stream has completed, so the launch just
 * before the call may write them.
 * Calls on one handle must be ordered on the device. */
moe_status moe_linear_forward(moe_linear_t linear, const void* x, int x_type, long long x_stride,
                              const float* x_scale, int T, const moe_w4* w,
                              const moe_lora* lora, const int32_t* adapter, uint16_t* y,
                              long long y_stride, moe_stream_t stream);

/* As moe_get_error, for a projection. */
moe_status moe_linear_get_error(moe_linear_t linear);

/* ------------------------------------------- attention over a paged cache ---
 * Keys and values of all requests lie in pages of one cache,
 *   k, v [pages][kv_heads][page_size][head_dim],
 * bf16, or e4m3 with a scale per key-value head (value = code * scale). Slot s
 * is row s % page_size of page s / page_size. A request's block table lists its
 * pages in the order of its tokens. */
typedef struct {
  void* k;
  void* v;
  const float* k_scale;    /* f32 [kv_heads], e4m3 only */
  const float* v_scale;
  int pages;
} moe_kv_cache;

/* Pages that requests own, and a ring of free ones. owned_out and ring_pos_out
 * may be owned and ring_pos themselves (the state is then updated in place) or
 * buffers that overlap nothing else. */
typedef struct {
  int32_t* table;          /* [requests][table_width] pages of each request, updated */
  int32_t* ring;           /* [ring_size] free pages, updated */
  const int32_t* owned;    /* [requests] pages of each request */
  int32_t* owned_out;
  const int32_t* ring_pos; /* [2]: first free entry of the ring, free pages */
  int32_t* ring_pos_out;
} moe_page_pool;

/* What a step's kernels need to know of its tokens. mask may be NULL where
 * mask_words is 0. */
typedef struct {
  int32_t* length;         /* [requests] tokens with this step's; 0: not served */
  int32_t* offsets;        /* [requests + 1] first row of each request */
  int32_t* slot;           /* [max_tokens] */
  int32_t* position;       /* [max_tokens] */
  uint64_t* mask;          /* [max_tokens][mask_words] */
  int32_t* status;         /* [5], below */
} moe_token_map;

typedef struct {
  int requests;            /* 1..4096 */
  int page_size;           /* 16, 32, 64, 128 or 256 tokens */
  int table_width;         /* pages per row of the table, 1..262144 */
  int max_tokens;          /* rows of the token arrays, 1..2^20 */
  int ring_size;           /* entries of the ring, 1..2^30 */
  int mask_words;          /* 64-bit words of a mask row, 0..4 */
} moe_page_desc;

/* One step of a batch, from lengths that only the device knows: request b holds
 * context[b] tokens and adds added[b] new ones; added[b] < 0 ends it.
 *   - Token rows lie request after request: offsets[b] = sum of added before b,
 *     at most max_tokens.
 *   - A request that lacks pages takes them from the ring, in the order of the
 *     requests. It is served if its arguments are sound (context[b] >= 0 and in
 *     its pages, 0 <= owned[b] <= table_width, length within table_width pages,
 *     rows within max_tokens, with masks at most 64 * mask_words new tokens) and
 *     the ring holds its pages and those of all sound requests before it; else
 *     its length is 0, its pages stay and it takes none.
 *   - An ended request gives its pages to the ring's end, where all of them
 *     fit; they can be taken from the next call on. Its length is 0.
 *   - Row i of a served request has slot (context + i)'s and position context +
 *     its depth. parent NULL: a chain, depth i. parent [rows]: each new token's
 *     parent among the request's earlier new tokens (0..i-1) or -1, below the
 *     context; depth is the number of ancestors. mask: bits of the ancestors and
 *     the token itself, bit j for new token j.
 *   - Rows of requests that are not served, and rows behind the last request
 *     (up to max_tokens), get slot -1, position 0 and an empty mask.
 *   - status: rows, pages taken, requests refused, pages lacking, and rows whose
 *     parent is no earlier token (these count as -1).
 * parent needs mask_words >= 1. All arrays 4-byte aligned, mask 8. No two of
 * the written arrays overlap, nor a written one and one that is read but for
 * the pairs named above; table and ring are both. Calls on one pool are ordered on the
 * device. The new tokens of a tree have the slots of their rows: whoever accepts a path
 * of it whose rows are not consecutive moves its keys and values, or stores them again,
 * before the next step counts them as context. Needs no handle; runs on the current
 * device. */
moe_status moe_page_map(const moe_page_desc* desc, const int32_t* context, const int32_t* added,
                        const int32_t* parent, const moe_page_pool* pool, const moe_token_map* out,
                        moe_stream_t stream);

typedef enum { MOE_CACHE_BF16 = 0, MOE_CACHE_E4M3 = 1 } moe_cache_type;
/* Which elements of a head turn together: i and i + rotary_dim / 2, or 2i and
 * 2i + 1. */
typedef enum { MOE_ROPE_HALF = 0, MOE_ROPE_INTERLEAVED = 1 } moe_rope_layout;
/* Frequencies f_i = theta^(-2i / rotary_dim) for long contexts: as they are,
 * all divided by `factor`, or by parts: with r = original f_i / 2 pi turns within
 * the original length and g = clamp((r - low) / (high - low), 0, 1),
 * f_i (g + (1 - g) / factor). The ramp is over the turns; a checkpoint whose ramp is over
 * the pair's index between two rounded ends has other frequencies (up to 41% at theta
 * 10000, original 32768, low 1, high 32, factor 4 and 64 elements that turn), which this
 * does not give. */
typedef enum { MOE_ROPE_PLAIN = 0, MOE_ROPE_LINEAR = 1, MOE_ROPE_BY_PARTS = 2 } moe_rope_scaling;

typedef struct {
  int heads;               /* query heads, a multiple of kv_heads, at most 128 of them each */
  int kv_heads;            /* 1..256 */
  int head_dim;            /* 64, 128 or 256 */
  int page_size;           /* 16, 32, 64, 128 or 256 */
  int cache_type;          /* moe_cache_type */
  int max_tokens;          /* 1..2^20 */
  int max_requests;        /* 1..4096 */
  float softmax_scale;     /* 0: 1 / sqrt(head_dim) */
  int rotary_dim;          /* leading elements of a head that turn: 0..head_dim, a multiple of 16 */
  int rope_layout;         /* moe_rope_layout */
  int rope_scaling;        /* moe_rope_scaling */
  double rope_theta;
  double rope_factor, rope_low, rope_high;   /* factor >= 1, low < high */
  int rope_original;
  float rope_gain;         /* factor of cosine and sine; 0: 1 */
  int wait_limit_ms;       /* device bounded-wait limit (default 1000 if 0) */
} moe_attn_desc;

/* The attention of one layer shape: its frequencies, and scratch for sums of
 * rows that several SMs share. Calls on one handle must be ordered on the
 * device (two captured graphs that share a handle do not run at once); layers
 * of one shape may share a handle. Calls work on the handle's device, whatever
 * the current one; `stream` belongs to it. */
typedef struct moe_attn* moe_attn_t;

moe_status moe_attn_create(const moe_attn_desc* desc, int device, moe_attn_t* out);
moe_status moe_attn_destroy(moe_attn_t attn);
moe_status moe_attn_scratch_bytes(const moe_attn_desc* desc, size_t* bytes);

/* Rotary positions of T rows of queries [heads][head_dim] and keys, and the
 * store of keys and values [kv_heads][head_dim]:
 *   (a, b) -> gain (a cos - b sin, b cos + a sin), angle position[t] f_i,
 * the angle taken modulo a turn as a 64-bit fixed-point fraction, of frequencies in
 * double precision: right to 2^-24 of a turn at the ends of int32, and to 2^-26 (the
 * FP32 argument of sine and cosine) for positions up to 2^29. Keys and values go to slot[t] of the cache, each rounded once (e4m3: the value over its
 * head's scale, clamped to +-448, a NaN kept); a slot outside the cache stores
 * nothing. Two rows of one call with the same slot leave a mixture of theirs.
 * Row strides in elements, 0 = dense; multiples of 8, and q, k, v, q_out 16-byte
 * aligned (so q, k and v may be parts of one projection's rows). q_out may be q
 * with the same stride; otherwise it overlaps no input. */
moe_status moe_rope_store(moe_attn_t attn, const uint16_t* q, long long q_stride, const uint16_t* k,
                          long long k_stride, const uint16_t* v, long long v_stride, int T,
                          const int32_t* position, const int32_t* slot, uint16_t* q_out,
                          long long out_stride, const moe_kv_cache* cache, moe_stream_t stream);

/* Attention of new tokens over their requests' keys, the new ones included:
 * request b has rows offsets[b]..offsets[b+1]-1 (n of them), keys 0..length[b]-1
 * in the pages table[b], and context c = length[b] - n. Its row i sees key j if
 *   j < c, or j - c <= i and (mask NULL or bit j - c of the row's mask).
 *   out[t][h] = softmax(scale q[t][h] K^T over the keys seen) V  (bf16, rounded once)
 * Offsets ascend. Key-value head h / (heads / kv_heads) serves query head h. mask: [T][mask_words],
 * mask_words 1..4; new tokens past 64 * mask_words have no bit and are not seen.
 * A row that sees no key, or none whose score is above -infinity, is zero, and so is
 * every row of a request with length[b] < n.
 * Rows before offsets[0] and from offsets[requests] on are left as they were.
 * Keys and values that no row sees may hold anything; what a row does not see
 * does not reach it, an infinity or a NaN neither. Rows from T on are not there
 * (n counts them, so the others keep their context and results), offsets below 0
 * count as 0, and lengths go up to table_width pages; a longer length, and a table
 * entry outside the cache, sets MOE_ERR_OPERAND_RANGE for moe_attn_get_error (the length is cut,
 * the page read as zeros). Scores, softmax and sums are FP32; the weights of V
 * are rounded to bf16, with an e4m3 cache to fp16 instead, in steps of 2^-31 of a
 * row's largest for weights below 2^-21 of it; those below 2^-32 count as zero. With an e4m3 cache a row's queries are
 * kept exactly down to 2^-9 of its largest element, smaller ones to 2^-17 of it,
 * and an infinity among them counts as a NaN; scales are positive and finite.
 * q_stride a multiple of 8, out_stride at least heads *
 * head_dim and a multiple of 8; q, out and the cache 16-byte aligned. out overlaps
 * no input. The result of a row does not depend on which other rows are in the
 * call but for the order of its sums. */
moe_status moe_tree_attention(moe_attn_t attn, const uint16_t* q, long long q_stride, int T,
                              const moe_kv_cache* cache, const int32_t* table, int table_width,
                              int requests, const int32_t* offsets, const int32_t* length,
                              const uint64_t* mask, int mask_words, uint16_t* out,
                              long long out_stride, moe_stream_t stream);

/* As moe_get_error, for an attention handle. */
moe_status moe_attn_get_error(moe_attn_t attn);

/* Reads and clears the plan's device error word. Synchronises the device:
 * call it between layers or steps, never inside one. Returns MOE_OK,
 * MOE_ERR_DEVICE_TIMEOUT (a bounded wait ran out; reported first),
 * MOE_ERR_OPERAND_RANGE (an input outside the fp16 operand contract above),
 * or MOE_ERR_CUDA if the context has failed. */
moe_status moe_get_error(moe_plan_t plan);

/* Launch a kernel whose bounded wait can never be satisfied, with the given
 * limit: it must give up, latch MOE_ERR_DEVICE_TIMEOUT and exit. Lets a test
 * check the failure path without faulting or hanging the GPU. */
moe_status moe_debug_wait_timeout(moe_plan_t plan, int limit_us, moe_stream_t stream);

/* Kernel timing for profiling. When enabled, every kernel the plan launches
 * is bracketed by CUDA events on its stream. moe_read_timing synchronises,
 * adds up the elapsed times per kernel kind since the last read, and resets.
 * Kinds: 0 router logits, 1 scan, 2 scatter, 3 gather, 4 gate/up GEMM,
 * 5 down GEMM, 6 combine, 7 residual, 8 top-k selection, 9 fused decode
 * layer. */
#define MOE_NUM_KERNEL_KINDS 10
typedef struct {
  double ms[MOE_NUM_KERNEL_KINDS];
  long long launches[MOE_NUM_KERNEL_KINDS];
} moe_timing;
moe_status moe_enable_timing(moe_plan_t plan, int on);
moe_status moe_read_timing(moe_plan_t plan, moe_timing* out);

/* Introspection of plan scratch for tests and profiling: device address of
 * the gathered activations (which = 0: fp16 [rows][H], routed positions
 * first, then the shared expert's T rows), the SwiGLU activations (1: fp16
 * [rows][I]) -- both with each block of 8 columns stored in the order
 * (0,4,1,5,2,6,3,7) --, the weighted routed expert outputs (2: bf16 [T*k][H]) or the
 * shared expert's outputs (3: f32 [T][H]) of the last layer. NULL for an
 * unknown `which` or a plan without a shared expert (3). */
void* moe_debug_buffer(moe_plan_t plan, int which);

/* Which GEMM path the last layer call took: 1 tensor-core, 2 small-M, 3 the
 * fused decode layer of moe_forward_stack, 4 tensor-core on SM pairs. */
int moe_last_gemm_path(moe_plan_t plan);

/* Load balance of the tensor-core path for expert groups of very different
 * sizes (the grouped GEMM of section "Las optimizaciones en el prefill"
 * runs over groups whose sizes vary by expert); on = 1, off = 0 (the
 * default). Units (one
 * 128-token tile x one weight block pair) are dealt in rounds over the SMs,
 * and when the last round holds at most half as many units as SMs, each of
 * its units is cut along K into two halves on different SMs, whose fp32
 * partial sums the SM that finishes second adds (one addition, the same
 * bits whichever SM that is: the result is the same on every run).
 * A token's output then depends, in its last bits, on whether its tile fell
 * into the last round. Off, every tile is summed over K in one pass, so a
 * prompt run in chunks gives the bits of one pass. Off by default: on the
 * 2048- and 4096-token workloads the split measured slower (the halves'
 * partial sums cost more than the idle SMs of the last round). Host only;
 * takes effect from the next call. */
moe_status moe_set_tail_split(moe_plan_t plan, int on);

/* Text of a status code. */
const char* moe_status_string(moe_status s);

/* Library version, major*10000 + minor*100 + patch. */
int moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_W4_H */
