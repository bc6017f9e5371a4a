/*
 * moe.h -- C ABI of the B200 routed mixture-of-experts FFN computed from low-bit blocks.
 *
 * The operation (one layer, per token t with input x_t of d_model values):
 *   logits = Wr x_t + b                       router over n_experts experts
 *   S      = the top_k largest logits (equal logits: lower expert index first)
 *   w_j    = softmax of the selected logits (fp32)
 *   o_e    = Wd_e (silu(Wg_e x_t) * (Wu_e x_t))   SwiGLU expert FFN, silu(z) = z sigmoid(z)
 *   y_t    = sum_{j in S} w_j o_j + o_shared(x_t)
 * Variants (moe_config): a selection-only router bias (bias_mode) and a sigmoid-gated shared
 * expert (shared_gate), y_t = sum_j w_j o_j + sigmoid(g . x_t) o_shared(x_t).
 * A stack applies layers first..first+n-1 with a residual add, x <- x + y, kept in fp32.
 * Sources: the hao.cnyes.com Strata feature article, "Strata 到底是什麼" (48 layers x 512
 * experts, about 10 routed per token) and its section 1 (router and shared expert always
 * resident); the strata-mlx README, "The file as it is" (experts stay in the file's low-bit
 * blocks and are multiplied from them), "Draft and verify" (1 + 7 token verify passes) and
 * "Prompts" (prompts read in chunks, experts a tile at a time on matrix hardware).
 *
 * Weight blocks (32 weights each, along a matrix row = the reduction dimension):
 *   MOE_FMT_Q2_32   10 B: fp16 scale s (LE), 8 B of 2-bit codes q (weight i: byte i/4, bits
 *                   2*(i%4)); w = s * (q - 1.5)
 *   MOE_FMT_CB35_32 14 B: fp16 scale s, 8 index bytes (byte g: grid row of weights 4g..4g+3),
 *                   uint32 LE sign mask (bit i negates weight i); w = s * sign * grid[row][i%4]
 *   MOE_FMT_NVFP4_16 9 B per 16 weights: FP8 E4M3 block scale s, 16 FP4 E2M1 codes (weight i
 *                   in byte 1 + i/2, low nibble for even i); each matrix starts with a 4-byte LE
 *                   fp32 tensor scale g; w = g * s * e2m1(code)  (hao.cnyes.com, the supported
 *                   models list: an NVIDIA-only NVFP4 file)
 * An expert's bytes are [gate: d_ff x d_model][up: d_ff x d_model][down: d_model x d_ff],
 * each row-major in blocks; routed experts are contiguous in index order.
 *
 * Conventions
 *  - Every call returns a moe_status.  Argument errors are detected synchronously.
 *  - Work is enqueued on the caller's CUDA stream (passed as void*, a cudaStream_t; NULL =
 *    the legacy default stream).  moe_forward / moe_forward_stack never synchronise the host
 *    when x and y are device pointers.
 *  - Pointers marked "host or device" are classified with cudaPointerGetAttributes; host
 *    buffers are staged through library-owned device memory (the call then completes before
 *    it returns).
 *  - The caller owns every buffer it passes.  The library owns the handle, the repacked
 *    weights and its workspace; moe_destroy frees them after a device synchronisation.
 *  - One handle serves one stream at a time (its workspace is shared by its calls).
 *  - Device-side failures (a bounded wait that ran out, a bad routing index) set an error
 *    word in host-mapped memory; the next call on the handle (or moe_check) returns
 *    MOE_ERR_TIMEOUT / MOE_ERR_DEVICE_FAULT and clears it.
 */
#ifndef EXPERT_FFN_GEMV_B200_MOE_H
#define EXPERT_FFN_GEMV_B200_MOE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARGUMENT = 1,
  MOE_ERR_OUT_OF_MEMORY = 2,
  MOE_ERR_CUDA = 3,
  MOE_ERR_NOT_LOADED = 4,
  MOE_ERR_UNSUPPORTED = 5,
  MOE_ERR_TIMEOUT = 6,
  MOE_ERR_DEVICE_FAULT = 7
} moe_status;

typedef enum { MOE_FMT_Q2_32 = 0, MOE_FMT_CB35_32 = 1, MOE_FMT_NVFP4_16 = 2 } moe_format;
typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;
/* How the router bias enters: MOE_BIAS_LOGIT adds b to the logits used for the selection and for
 * the weights (the plain definition above); MOE_BIAS_SELECT selects the top_k of (logit + b) and
 * weighs them by the softmax of their unbiased logits (a bias that only balances expert load). */
typedef enum { MOE_BIAS_LOGIT = 0, MOE_BIAS_SELECT = 1 } moe_bias_mode;

typedef struct moe_handle moe_handle; /* opaque */

typedef struct {
  uint32_t struct_size;   /* sizeof(moe_config): ABI version check */
  int32_t n_layers;       /* layers the handle can hold, >= 1 */
  int32_t d_model;        /* D, multiple of 128, at most 4096 */
  int32_t d_ff;           /* F of routed experts, multiple of 128, at most 1024 */
  int32_t n_experts;      /* E, 1..4096 */
  int32_t top_k;          /* k, 1..min(E, 32) */
  int32_t n_shared;       /* 0 or 1 shared expert (weight 1, always applied) */
  int32_t shared_d_ff;    /* F of the shared expert, multiple of 128, at most 1024 (ignored if
                             n_shared = 0) */
  int32_t fmt;            /* moe_format */
  int32_t act_dtype;      /* dtype of x given to moe_forward / moe_forward_stack */
  int32_t router_dtype;   /* dtype of the router weight rows */
  int32_t out_dtype;      /* dtype of y / x_out */
  int32_t max_tokens;     /* largest n_tokens per call, 1..8192: sizes the workspace */
  const int8_t *codebook_grid; /* host, 256 x 4 int8, copied at create; required iff CB35 */
  int32_t device;         /* CUDA device ordinal */
  int32_t bias_mode;      /* moe_bias_mode */
  int32_t shared_gate;    /* 1: o_shared is scaled by sigmoid(g . x_t), g a d_model vector given
                             per layer (requires n_shared = 1); 0: weight 1 */
} moe_config;

typedef struct {
  const void *router_w;      /* host or device: n_experts x d_model, router_dtype, row-major */
  const float *router_bias;  /* host or device: n_experts fp32, or NULL (= 0) */
  const void *expert_blocks; /* host or device: n_experts experts, interchange bytes (above) */
  const void *shared_blocks; /* host or device: the shared expert; NULL iff n_shared == 0 */
  const void *shared_gate_w; /* host or device: d_model values g (router_dtype); required iff
                                cfg.shared_gate, else ignored */
} moe_layer_weights;

typedef struct {             /* device pointers, each may be NULL */
  int32_t *topk_idx;         /* n_tokens x top_k expert ids, descending router logit */
  float *topk_w;             /* n_tokens x top_k routing weights (sum to 1 per token) */
  int32_t *expert_counts;    /* n_experts: tokens routed to each expert in this call */
} moe_route_out;

/* Create a handle on cfg->device: validates cfg, allocates the workspace for max_tokens.
 * Errors: INVALID_ARGUMENT (bad or inconsistent cfg, NULL out), OUT_OF_MEMORY, CUDA. */
moe_status moe_create(const moe_config *cfg, moe_handle **out);

/* Copy one layer's weights into library-owned HBM, repacked on the device into tiled planes
 * (same bits per weight, nothing dequantised).  Enqueued on `stream`; the sources may be
 * reused once the stream passes this point (host sources: when the call returns).
 * Reloading a layer replaces it.  Errors: INVALID_ARGUMENT, OUT_OF_MEMORY, CUDA. */
moe_status moe_load_layer(moe_handle *h, int32_t layer, const moe_layer_weights *w, void *stream);

/* One layer: y = MoE_layer(x) (no residual).  x: host or device, n_tokens x d_model in
 * act_dtype; y: host or device, n_tokens x d_model in out_dtype.  n_tokens in 1..max_tokens:
 * up to 8 tokens run the dequant-fused GEMV path (decode / verify batches), more run the
 * grouped tensor-core path (prompt chunks).  route: optional device outputs for this call.
 * Errors: INVALID_ARGUMENT, NOT_LOADED, CUDA, TIMEOUT / DEVICE_FAULT (from an earlier call). */
moe_status moe_forward(moe_handle *h, int32_t layer, const void *x, void *y, int32_t n_tokens,
                       void *stream, moe_route_out *route);

/* Layers first_layer .. first_layer + n_layers - 1 with x <- x + MoE_l(x) after each, the
 * residual stream in fp32.  x_in: act_dtype, x_out: out_dtype (host or device, may not
 * alias).  per_layer_route: NULL or an array of n_layers moe_route_out.  x_trace: NULL or a
 * device fp32 buffer of n_layers x n_tokens x d_model receiving each layer's input. */
moe_status moe_forward_stack(moe_handle *h, int32_t first_layer, int32_t n_layers,
                             const void *x_in, void *x_out, int32_t n_tokens, void *stream,
                             moe_route_out *per_layer_route, float *x_trace);

/* Return (and clear) a pending device-side error of the handle without enqueuing work. */
moe_status moe_check(moe_handle *h);

/* Free everything owned by the handle (after a device synchronisation).  NULL is a no-op. */
moe_status moe_destroy(moe_handle *h);

/* Static description of a status code. */
const char *moe_status_string(moe_status s);

/* Detail of the last failure on this handle ("" if none; a static string if h is NULL). */
const char *moe_last_error(const moe_handle *h);

/* Bytes of device memory held by the handle (weights + workspace). */
uint64_t moe_device_bytes(const moe_handle *h);

/* Per-kernel CUDA-event timing.  While enabled (on != 0), every forward call records an event
 * pair on its stream around the launches of each selected kernel class of each layer it runs
 * (bit k of `on` selects class k; such events are captured into a CUDA graph like the kernels).
 * moe_profile_read sums, over the layers run since profiling was (re-)enabled, the durations
 * recorded by the latest call that ran each layer, for one kernel class -- 0: router + top-k
 * (+ grouping); 1: the expert matrices (1-8 tokens: the one GEMV kernel that runs gate/up +
 * SwiGLU and down; more tokens: the gate/up GEMM + SwiGLU); 2: what follows (1-8 tokens: the
 * weighted combine; more tokens: the down GEMM + combine) -- and returns how many layers
 * contributed.  It waits for those events to complete. */
moe_status moe_profile_enable(moe_handle *h, int32_t on);
moe_status moe_profile_read(moe_handle *h, int32_t kind, float *total_ms, int32_t *launches);

/* Routing without a handle and without any device allocation.  Some callers cannot allocate
 * device memory at the point where they route: runtimes that plan every byte of device memory
 * up front and pass kernels only the buffers they planned, and loops that must not take the
 * device-wide synchronisation that cudaMalloc / cudaFree can imply.  This entry point has no
 * counterpart in the paper: it is the routing step of moe_forward (router logits with fp32
 * accumulation, top-k with equal logits resolved to the lower expert index and NaN logits taken
 * after every numeric one, fp32 softmax over the selected logits) without a handle.
 * All pointers are device pointers on the current device: router_w n_experts x d_model
 * (router_dtype, row-major, 16-byte aligned: it is read 16 bytes at a time), router_bias
 * n_experts fp32 or NULL, x n_tokens x d_model (x_dtype); outputs topk_idx / topk_w
 * n_tokens x top_k, descending logit.  A selected -inf (or NaN) logit gets weight 0; a token whose
 * largest selected logit is not finite gets NaN weights.
 * It allocates nothing: its scratch (the logits and an arrival counter, 32 KB) is a file-scope
 * device array that every GPU loading the library holds until the process exits.  The first call
 * on a device looks up that array's device address and sets the kernel's shared-memory limit;
 * make that first call before any stream capture.  Limits: n_tokens <= 8, n_experts <= 1024,
 * d_model <= 4096 (a multiple of 128), top_k <= 32; larger sizes return MOE_ERR_UNSUPPORTED,
 * malformed arguments (NULL, out of range, a misaligned router_w) MOE_ERR_INVALID_ARGUMENT.
 * Every call shares the one array and leaves its contents behind (the arrival counter is cleared
 * on the stream before each launch); calls whose kernels may overlap on one device race on it,
 * so keep them in one stream order. */
moe_status moe_route_noalloc(const void *router_w, int32_t router_dtype, const float *router_bias,
                             int32_t n_experts, int32_t d_model, int32_t top_k, const void *x,
                             int32_t x_dtype, int32_t n_tokens, int32_t *topk_idx, float *topk_w,
                             void *stream);

/* ---------------------------------------------------------------------------------------------
 * Block operators: what stands around and beside the routed experts in a transformer layer.  Norms
 * before and after a block with gate and residual scale, low-rank adapters of many requests, and a
 * dense gated feed-forward block from bf16 weights (a layer, or a shared block, that is not kept
 * in low-bit blocks), with the gradients of the norms and of the dense block (they are local to a
 * layer, so a quantised layer can be tuned against its original with the routed experts frozen).
 * All of them take device pointers, run on the current device (adapters: on their handle's),
 * enqueue on `stream`, never synchronise the host and allocate nothing, so they can be captured
 * into a CUDA graph (after a first call outside a capture, which loads and configures kernels and
 * pins a page of host memory for error words).  Strides count values between the starts of
 * consecutive rows.  Calls with the same inputs give the same bits.
 *
 * Sums, norms and accumulators are held in fp32 and each result is rounded once to its type.  Three
 * things inside are held to less than fp32:
 *   - the dense block's hidden values, and in its backward the gradients of its gate and up products,
 *     are bf16 between the products, as operands of the tensor cores: half a step is up to 2^-8 of a
 *     value, and bf16 results are 2.4e-3 off in place of 1.7e-3 (relative 2-norm, against 64 bits);
 *   - fp32 x and the low-rank values of the adapters enter bf16 products as parts: exactly where out
 *     is fp32, to 2^-16 of a value where it is bf16;
 *   - SiLU and the sigmoids of gates by the value (channel, full) use approximate instructions: an
 *     argument z costs up to (1.25 |z| + 7) 2^-24, relative.  A token's gate takes expf and a division.
 * Outputs may not overlap inputs unless said so; one in an input's place that has another type or
 * row stride is refused.
 * ------------------------------------------------------------------------------------------- */
/* A bounded wait of the norms' or the dense block's kernels that ran out makes the next call of one of
 * them on that device, whoever made the first, return MOE_ERR_TIMEOUT, once and with nothing launched:
 * the results of an earlier call are not valid.  moe_block_check waits for the current device, all its
 * streams, and returns (and clears) what is pending there. */
moe_status moe_block_check(void);

/* What a gate is broadcast over: one value per column, per token, or of its own for every value. */
typedef enum { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_TOKEN = 2, MOE_GATE_FULL = 3 } moe_gate_kind;
/* a(g) = g, or sigmoid(g) */
typedef enum { MOE_GATE_LINEAR = 0, MOE_GATE_SIGMOID = 1 } moe_gate_act;

/* Norm before a block: h_t = x_t / sqrt(mean(x_t^2) + eps) * (weight + unit_offset).
 * x, h: n_tokens x d_model (x_dtype, h_dtype); h may be x when types and strides agree.
 * d_model 1..8192 (larger: UNSUPPORTED), n_tokens >= 1, eps >= 0, unit_offset 0 or 1. */
moe_status moe_norm_in(const void *x, int32_t x_dtype, int64_t x_stride, const void *weight, int32_t w_dtype, float eps,
                       int32_t unit_offset, void *h, int32_t h_dtype, int64_t h_stride, int32_t n_tokens,
                       int32_t d_model, void *stream);

/* Norm after a block, its gate, the residual scale and add, and (h != NULL) the next block's input
 * norm in the same pass:
 *   u = o / sqrt(mean(o^2) + eps) * (weight + unit_offset)      (weight NULL: u = o)
 *   res_out = residual + scale * a(gate) * u                    (no gate: a = 1)
 *   h = res_out / sqrt(mean(res_out^2) + next_eps) * (next_weight + unit_offset)
 * h is computed from res_out as it is stored, so it equals moe_norm_in of res_out.  res_out may be
 * residual or o, and h may be o, when types and strides agree. */
typedef struct {
  uint32_t struct_size;      /* sizeof(moe_norm_out_args) */
  int32_t n_tokens, d_model;
  int32_t o_dtype, res_dtype, res_out_dtype, w_dtype, gate_dtype, h_dtype; /* moe_dtype */
  int32_t gate_kind, gate_act, unit_offset;
  float eps, next_eps, scale;
  const void *o;             /* n_tokens x d_model: the block's output */
  const void *residual;      /* n_tokens x d_model */
  const void *weight;        /* d_model, w_dtype, or NULL */
  const void *gate;          /* by gate_kind: d_model; n_tokens; n_tokens x d_model; NULL */
  void *res_out;             /* n_tokens x d_model */
  const void *next_weight;   /* d_model, w_dtype; NULL iff h is NULL */
  void *h;                   /* n_tokens x d_model, or NULL */
  int64_t o_stride, res_stride, gate_stride, res_out_stride, h_stride; /* gate: token and full */
} moe_norm_out_args;
moe_status moe_norm_out(const moe_norm_out_args *args, void *stream);

/* Bytes of workspace that either backward call needs (0: sizes out of range). */
uint64_t moe_norm_workspace(int32_t n_tokens, int32_t d_model);

/* Gradients of moe_norm_in: dx = dres + (dh's gradient through the norm), dweight = sum over tokens.
 * dres (or NULL): a gradient that reaches x another way, e.g. over the residual; dx may be dres. */
typedef struct {
  uint32_t struct_size;
  int32_t n_tokens, d_model;
  int32_t x_dtype, w_dtype, dh_dtype, dres_dtype, dx_dtype, unit_offset;
  float eps;
  const void *x, *weight, *dh, *dres;
  void *dx;
  void *dweight;             /* d_model, w_dtype, or NULL */
  void *workspace;           /* 16-byte aligned; not needed when dweight is NULL */
  uint64_t workspace_bytes;
  int64_t x_stride, dh_stride, dres_stride, dx_stride;
} moe_norm_in_bwd_args;
moe_status moe_norm_in_backward(const moe_norm_in_bwd_args *args, void *stream);

/* Gradients of moe_norm_out (without h) from dres = the gradient of res_out, which is the gradient
 * of residual as it stands: d_o (o_dtype), dweight and dgate (the gate's shape and type; dgate_stride
 * for token and full). */
typedef struct {
  uint32_t struct_size;
  int32_t n_tokens, d_model;
  int32_t o_dtype, w_dtype, gate_dtype, dres_dtype;
  int32_t gate_kind, gate_act, unit_offset;
  float eps, scale;
  const void *o, *weight, *gate, *dres;
  void *d_o;
  void *dweight;             /* or NULL */
  void *dgate;               /* or NULL */
  void *workspace;           /* 16-byte aligned; for dweight and a channel gate's dgate */
  uint64_t workspace_bytes;
  int64_t o_stride, gate_stride, dres_stride, do_stride, dgate_stride;
} moe_norm_out_bwd_args;
moe_status moe_norm_out_backward(const moe_norm_out_bwd_args *args, void *stream);

/* Low-rank adapters of many requests:  out_t = base_t + scale_i B_i (A_i x_t) with i = ids[t], and
 * out_t = base_t where ids[t] = -1.  The handle owns the adapters (repacked).  moe_adapters_apply
 * writes nothing but out, so calls of one handle may run at once on several streams and in captured
 * graphs; a load is ordered by its stream, and loads are made one at a time. */
typedef struct moe_adapters moe_adapters; /* opaque */
typedef struct {
  uint32_t struct_size;   /* sizeof(moe_adapters_config) */
  int32_t d_in, d_out;    /* multiples of 8, 8..65536 */
  int32_t max_adapters;   /* slots, 1..4096 */
  int32_t max_rank;       /* 1..128 */
  int32_t max_tokens;     /* largest n_tokens per call, 1..8192 */
  int32_t device;
} moe_adapters_config;
moe_status moe_adapters_create(const moe_adapters_config *cfg, moe_adapters **out);
/* Put an adapter into a slot (replacing what is there, in stream order): a rank x d_in and b
 * d_out x rank, bf16, row-major, host or device (host sources: the call waits for the copy).
 * rank 0 (a, b NULL) empties the slot. */
moe_status moe_adapters_load(moe_adapters *h, int32_t slot, const void *a, const void *b, int32_t rank, float scale,
                             void *stream);
/* x: n_tokens x d_in (x_dtype); base, out: n_tokens x d_out (out_dtype); out may be base (same
 * stride), then rows without an adapter are not touched.  ids: n_tokens slots on the device.
 * Pointers and row strides must be multiples of 16 bytes.  An id that is out of range or names an
 * empty slot counts as -1 and makes the next call (or moe_adapters_check) return
 * MOE_ERR_DEVICE_FAULT. */
moe_status moe_adapters_apply(moe_adapters *h, const void *x, int32_t x_dtype, int64_t x_stride, const void *base,
                              int64_t base_stride, void *out, int64_t out_stride, int32_t out_dtype, const int32_t *ids,
                              int32_t n_tokens, void *stream);
moe_status moe_adapters_check(moe_adapters *h);
moe_status moe_adapters_destroy(moe_adapters *h);
const char *moe_adapters_last_error(const moe_adapters *h);
uint64_t moe_adapters_device_bytes(const moe_adapters *h);

/* Dense gated feed-forward block, bf16 weights: y = w_down (silu(w_gate x) * (w_up x)) (+ add).
 * n_tokens 1..1048576; d_model and d_ff: multiples of 8, 8..65536; every pointer 16-byte aligned, every row stride a
 * multiple of 16 bytes.  The hidden values are kept in bf16 between the products (the pre-activations, if
 * saved, in fp32). */
typedef struct {
  uint32_t struct_size;
  int32_t n_tokens, d_model, d_ff;
  int32_t add_dtype, y_dtype;
  const void *x;                       /* n_tokens x d_model, bf16 */
  const void *w_gate, *w_up, *w_down;  /* d_ff x d_model, d_ff x d_model, d_model x d_ff, bf16 */
  const void *add;                     /* n_tokens x d_model added to the result, or NULL; may be y */
  void *y;                             /* n_tokens x d_model */
  void *save_gate, *save_up;           /* for the backward: w_gate x and w_up x, n_tokens x d_ff
                                          fp32, or both NULL */
  void *workspace;                     /* moe_ffn_workspace(.., 0) bytes, used by one call at a time */
  uint64_t workspace_bytes;
  int64_t x_stride, add_stride, y_stride;
} moe_ffn_args;
uint64_t moe_ffn_workspace(int32_t n_tokens, int32_t d_model, int32_t d_ff, int32_t backward);
moe_status moe_ffn_forward(const moe_ffn_args *args, void *stream);

/* Its gradients from dy (of the block alone: the gradient of add is dy itself).  All outputs bf16; the
 * gradients of the gate and up products, operands of all of them, are bf16 too, and h is made again in bf16.
 * dx, the pair dw_gate / dw_up and dw_down may each be NULL, not all of them. */
typedef struct {
  uint32_t struct_size;
  int32_t n_tokens, d_model, d_ff;
  const void *dy, *x;                  /* n_tokens x d_model, bf16 */
  const void *w_gate, *w_up, *w_down;
  const void *save_gate, *save_up;     /* of the forward call */
  void *dx;                            /* n_tokens x d_model */
  void *dw_gate, *dw_up, *dw_down;     /* the weights' shapes */
  void *workspace;                     /* moe_ffn_workspace(.., 1) bytes */
  uint64_t workspace_bytes;
  int64_t dy_stride, x_stride, dx_stride;
} moe_ffn_bwd_args;
moe_status moe_ffn_backward(const moe_ffn_bwd_args *args, void *stream);
/* A run of layers first_layer .. first_layer + n_layers - 1 with everything that stands around and
 * beside their routed experts, x kept in fp32 between the layers:
 *   a = norm_in(x)            o = MoE_l(a) (+ dense block(a)) (+ adapters(a))
 *   x = x + scale * act(gate) * norm_out(o)
 * One moe_block per layer; the caller keeps what it points to (device memory) alive. */
typedef struct {
  uint32_t struct_size;      /* sizeof(moe_block) */
  int32_t norm_dtype;        /* of the norm weights and the gate */
  const void *norm_in_w;     /* d_model, required */
  const void *norm_out_w;    /* d_model, or NULL: no norm after the block */
  const void *gate;          /* d_model values (one per column), or NULL */
  float norm_in_eps, norm_out_eps, scale;
  int32_t gate_act, unit_offset;
  int32_t ffn_d_ff;          /* dense block beside the experts: its d_ff, 0: none */
  const void *ffn_gate, *ffn_up, *ffn_down;
  moe_adapters *adapters;    /* d_in = d_out = d_model, or NULL */
} moe_block;
/* Bytes of workspace for these blocks (0 when no layer has a dense block). */
uint64_t moe_blocks_workspace(const moe_handle *h, const moe_block *blocks, int32_t n_layers, int32_t n_tokens);
/* x_in: act_dtype, x_out: out_dtype, device memory, not aliased.  adapter_ids: n_tokens slots, or NULL
 * when no layer has adapters.  A dense block needs act_dtype = MOE_BF16.  Errors as
 * moe_forward_stack, and those of the operators; a bounded wait that runs out in any kernel of the run
 * but the adapters' is reported by the next call on h (or moe_check), not by moe_block_check.  What
 * the adapters' kernels of earlier calls reported is returned before anything is launched; an id that
 * is out of range in this run counts as -1 in all its layers and is reported by a later call. */
moe_status moe_forward_blocks(moe_handle *h, int32_t first_layer, int32_t n_layers, const moe_block *blocks,
                              const void *x_in, void *x_out, int32_t n_tokens, const int32_t *adapter_ids,
                              void *workspace, uint64_t workspace_bytes, void *stream, moe_route_out *per_layer_route);

/* Test hooks.  moe_debug_set_spin_limit: clock cycles a device-side bounded wait may spin
 * before it gives up (0 restores the default of about one second).  moe_debug_set_alloc_cap:
 * fail allocations that would take the handle above `bytes` (0 = no cap).
 * moe_debug_set_ring_spin_limit: the same limit for the bulk-copy rings of the norms over many rows
 * and of the adapters, process-wide, for the launches that follow; each block's first copies are then held back for four
 * times as long, so that the waits for them run out
 * (200 million cycles at most). */
moe_status moe_debug_set_spin_limit(moe_handle *h, uint64_t cycles);
moe_status moe_debug_set_alloc_cap(moe_handle *h, uint64_t bytes);
moe_status moe_debug_set_ring_spin_limit(uint64_t cycles);
/* Enqueue a kernel that waits, bounded by the spin limit, on a device flag that nothing sets:
 * it gives up, sets the error word, and the next call on h returns MOE_ERR_TIMEOUT.  Exercises
 * the device-side timeout path without faulting or hanging the GPU. */
moe_status moe_debug_wait_test(moe_handle *h, void *stream);

#ifdef __cplusplus
}
#endif
#endif
