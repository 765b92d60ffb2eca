/*
 * moe.h - C ABI of a routed mixture-of-experts (MoE) layer forward on one
 * NVIDIA GB300 (sm_103a).
 *
 * The layer, as the source pages describe it:
 *   gate      L = x W_g + b, one logit per expert
 *             (DeepSeek-V4 EP article, section 2.1)
 *   router    max-subtracted softmax, partial top-8, exact top-k; the lower
 *             expert id wins a tie (same article, section 3.2)
 *   dispatch  per-expert histogram, exclusive scan and a stable permutation
 *             that packs the routed rows contiguously by expert id - the
 *             single-GPU form of the expert-parallel all-to-all layout
 *             (same article, section 3.3; Deepseek-MoE sync-tax article,
 *             section 2.1), optionally as a per-token FP8 E4M3 payload
 *             (sync-tax article, section 3.1)
 *   FFN       per expert e: H = SiLU(X_e W1_e), Y = H W2_e ("L1 + Act + L2",
 *             DeepSeek V3/V4 parallel-strategy article, Waved-EP section)
 *   combine   out_t = sum_{j=0..k-1} w_tj * Y[pos(t, j)], in that order
 *             (sync-tax article, section 2.3)
 *
 * Conventions for every entry point
 * ---------------------------------
 *  - Pointers named as device pointers must point to device (or managed)
 *    memory of the current CUDA device. Host pointers are never accepted.
 *  - All tensors are dense, row-major, with no padding between rows.
 *  - Device pointers to activations, weights, payloads, H, Y and outputs must
 *    be 16-byte aligned; the workspace must be 256-byte aligned.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream). Every call is asynchronous on that stream: it only enqueues
 *    kernels, never allocates, frees or synchronises (except
 *    moe_get_device_error, which synchronises by design). The caller owns
 *    every buffer, including the workspace.
 *  - Calls return MOE_OK (0) or a negative moe_status. Argument errors are
 *    found on the host before anything is enqueued. Errors found by a kernel
 *    (an expert index or row position out of range, a device wait that ran
 *    past its bound) are recorded in the workspace's error word; the kernel
 *    skips the offending access instead of faulting. Read them with
 *    moe_get_device_error.
 *  - T = 0 is valid and produces empty outputs (counts/offsets are zeroed).
 */
#ifndef MOE_GB300_MOE_H_
#define MOE_GB300_MOE_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1,         /* null pointer, misaligned pointer, bad shape */
  MOE_ERR_UNSUPPORTED = -2,         /* valid but unsupported combination */
  MOE_ERR_WORKSPACE_TOO_SMALL = -3, /* ws_bytes below the size query's answer */
  MOE_ERR_LAUNCH = -4,              /* a CUDA runtime/driver call failed */
  MOE_ERR_BAD_INDEX = -5,           /* device: expert id or row position out of range */
  MOE_ERR_TIMEOUT = -6              /* device: a bounded wait gave up */
} moe_status;

/* ---- configuration ----------------------------------------------------- */
enum { MOE_DTYPE_F32 = 0, MOE_DTYPE_BF16 = 1 };

enum {
  /* softmax over all E logits, keep the k largest, divide them by their sum */
  MOE_ROUTER_RENORM = 0,
  /* exact softmax over the pre_k largest logits only; keep its first k
   * entries without renormalising (the partial top-8 router of the
   * DeepSeek-V4 EP article, section 3.2) */
  MOE_ROUTER_PREK_SOFTMAX = 1,
  /* node-limited top-k (DeepSeek V3/V4 parallel-strategy article, EP
   * section: a token's experts come from its best nodes only). The E experts
   * form n_group equal groups of consecutive ids; a group's score is the
   * mean softmax probability of its experts; the topk_group best groups are
   * kept (equal scores: lower group id first); the k largest logits among
   * the kept groups' experts are chosen (lower id first on ties) and
   * weighted as in MOE_ROUTER_RENORM. pre_k is validated but not used. */
  MOE_ROUTER_GROUP_LIMITED = 2,
  /* soft gating (Deepseek-MoE sync-tax article, section 3.3: Gumbel-Softmax
   * instead of hard top-k, every expert output weighted): with g the
   * caller's Gumbel samples (the `noise` argument, [T, E] fp32),
   * w[t, e] = softmax_e((L[t, e] + g[t, e]) / tau), max-subtracted; k must
   * equal E (at most 16) and slot j holds expert j. Every token goes to
   * every expert in token order, so dispatch writes only the layout and the
   * W1 GEMM reads x itself (no packed rows, no FP8 payload). */
  MOE_ROUTER_SOFT_GUMBEL = 3
};

typedef struct moe_config {
  int32_t T;           /* tokens, >= 0 */
  int32_t d;           /* hidden size, multiple of 64 */
  int32_t E;           /* experts, 1..256 */
  int32_t k;           /* experts per token, 1..min(E, pre_k, 8) */
  int32_t f;           /* expert FFN inner size, multiple of 64 */
  int32_t dtype;       /* MOE_DTYPE_F32 or MOE_DTYPE_BF16: x, W_g, W1, W2, H, out */
  int32_t router;      /* MOE_ROUTER_* */
  int32_t pre_k;       /* partial top-k width, k..min(8, E) (8 on the pages) */
  int32_t payload_fp8; /* dispatch rows as FP8 E4M3 + an fp32 scale per row (bf16
                        * only): 1 = per-token absmax scale; 2 = one static
                        * scale, payload_scale, for every row (the sync-tax
                        * article's "static global" variant, section 3.1) */
  int32_t n_group;     /* MOE_ROUTER_GROUP_LIMITED: expert groups, 1..32, dividing E;
                        * ignored by the other routers */
  int32_t topk_group;  /* MOE_ROUTER_GROUP_LIMITED: groups kept per token,
                        * 1..n_group, with k <= topk_group * E / n_group */
  float payload_scale; /* payload_fp8 == 2: the scale, finite and > 0; values
                        * beyond 448 * payload_scale saturate to +-448 */
  int32_t output_fp8;  /* 1: moe_forward hands the expert outputs to the combine
                        * as an FP8 payload (moe_quantize_output, then
                        * moe_combine_fp8); 0: fp32 rows (moe_combine) */
  float tau;           /* MOE_ROUTER_SOFT_GUMBEL: temperature, finite and > 0 */
  int32_t gemm_tile_n; /* bf16 expert GEMMs: output features per 2-SM pair tile.
                        * 0 = the library's choice (512 for long-K SiLU passes
                        * with many tiles, else 256); 256 or 512 force it (the
                        * FP8 payload's W1 pass always takes 256). A tuning
                        * knob with no effect on the result beyond fp32
                        * summation order; other values: MOE_ERR_INVALID_ARG */
  int32_t x_perm_mode; /* moe_forward's packed rows (MOE_XPERM_*): packed by the
                        * dispatch into x_perm and read by the W1 GEMM, or
                        * gathered by the W1 GEMM from x through src, x_perm
                        * never written (the dispatch and the first expert
                        * GEMM in one pass: the single-GPU form of the
                        * Waved-EP fusion, DeepSeek V3/V4 parallel-strategy
                        * article). Gathering takes bf16 layers without an FP8
                        * payload or soft gating; asking for it elsewhere is
                        * MOE_ERR_UNSUPPORTED. The stage calls always pack. */
  int32_t keep_z;      /* 1: moe_forward also keeps the W1 GEMM's pre-activation
                        * Z = X_e W1_e [T k, f] (fp32, the value SiLU takes) in
                        * its workspace (moe_workspace_size grows by T k f 4
                        * bytes), and moe_backward, given the same config,
                        * reads it there instead of recomputing it. For a
                        * forward followed by a backward (training); not
                        * with an FP8 payload (those have no backward):
                        * MOE_ERR_UNSUPPORTED. Other values than 0 and 1:
                        * MOE_ERR_INVALID_ARG */
} moe_config_t;

enum {
  MOE_XPERM_AUTO = 0,     /* the library's choice: gathered where it can be and
                           * the packed rows (T k d bf16 values) would take
                           * 256 MiB or more, else packed */
  MOE_XPERM_PACKED = 1,   /* the dispatch writes x_perm */
  MOE_XPERM_GATHERED = 2  /* the W1 GEMM reads x[src[r]]; no x_perm */
};

/* Validate a configuration. Returns MOE_OK or MOE_ERR_INVALID_ARG /
 * MOE_ERR_UNSUPPORTED without touching the device. */
MOE_API int moe_check_config(const moe_config_t* cfg);

/* ---- workspace ----------------------------------------------------------
 * moe_scratch_size: bytes of workspace that moe_dispatch, moe_expert_ffn and
 *   moe_combine need (an error word, the GEMM tile counters and the dispatch
 *   per-block tables).
 * moe_workspace_size: bytes moe_forward needs: the scratch above followed by
 *   every intermediate of the layer (routing, permutation, payload, H, Y).
 *   A forward workspace therefore also serves the stage calls.
 * Both return 0 for an invalid configuration. The caller allocates the
 * workspace (256-byte aligned); zero it once before first use, or call
 * moe_clear_device_error, so the error word starts clear. */
MOE_API size_t moe_scratch_size(const moe_config_t* cfg);
MOE_API size_t moe_workspace_size(const moe_config_t* cfg);

/* ---- stage 1: gate + router ---------------------------------------------
 * The gate's per-expert logit (DeepSeek-V4 EP article, section 2.1) and the
 * router's max-subtracted softmax, partial top-8 and exact top-k (section
 * 3.2); the variants as cited at moe_config.router.
 * x [T, d] (dtype), W_g [d, E] (dtype), bias [E] fp32 or NULL (= zeros),
 * noise [T, E] fp32: the Gumbel samples of MOE_ROUTER_SOFT_GUMBEL (required
 * there, ignored by the other routers, may be NULL).
 * Outputs: topk_idx [T, k] int32, topk_w [T, k] fp32, slot j = j-th choice
 * (logit descending, lower id first on ties; soft gating: expert j);
 * logits [T, E] fp32 or NULL: the gate logits including the bias, as the
 * router saw them (before the noise).
 * Logits are accumulated in fp32 from exact products, in K-chunks combined
 * with compensated summation. */
MOE_API int moe_route(const moe_config_t* cfg, const void* x, const void* W_g,
              const float* bias, const float* noise, int32_t* topk_idx, float* topk_w,
              float* logits, void* stream);

/* ---- stage 2: dispatch ---------------------------------------------------
 * Packing by expert id (DeepSeek-V4 EP article, section 3.3; Deepseek-MoE
 * sync-tax article, section 2.1), with the optional FP8 payload (sync-tax
 * article, section 3.1).
 * Inputs: x [T, d] (dtype), topk_idx [T, k] int32.
 * (MOE_ROUTER_SOFT_GUMBEL: only counts, offsets, pos and src are written,
 * for the routing every token -> every expert in token order; x, topk_idx,
 * x_perm and x_scale are not used and may be NULL.)
 * Outputs (R = T*k):
 *   counts  [E]    int32  rows routed to each expert
 *   offsets [E+1]  int32  exclusive prefix sum of counts; offsets[E] = R
 *   pos     [R]    int32  flat entry i = t*k + j goes to row pos[i]; within an
 *                         expert, rows follow increasing i (stable)
 *   src     [R]    int32  src[pos[i]] = i / k (token of each packed row)
 *   x_perm  [R, d]        packed rows: x[src[r]] in dtype, or with
 *                         cfg->payload_fp8 the FP8 E4M3 bytes (uint8) of
 *                         x / scale, rounded to nearest even, saturating
 *   x_scale [R]    fp32   FP8 only (else may be NULL): scale = fp32(absmax of
 *                         the token's row / 448), 1 for an all-zero row
 * Entries of topk_idx outside [0, E) are skipped (pos = -1) and flag
 * MOE_ERR_BAD_INDEX in the error word. ws: >= moe_scratch_size bytes. */
MOE_API int moe_dispatch(const moe_config_t* cfg, const void* x, const int32_t* topk_idx,
                 int32_t* counts, int32_t* offsets, int32_t* pos, int32_t* src,
                 void* x_perm, float* x_scale, void* ws, size_t ws_bytes,
                 void* stream);

/* ---- dispatch without a workspace ---------------------------------------
 * The source pages have no counterpart to this entry point; it exists for
 * callers that cannot allocate device memory when they dispatch (a locked,
 * pre-sized memory pool; a plugin that is only handed its input and output
 * buffers; code that must not call cudaMalloc because it can synchronise
 * the device). It does what moe_dispatch does, with the same arguments
 * except the workspace: its scratch tables live in a fixed array compiled
 * into the library (4 MiB + 256 bytes, held on every GPU that loads the
 * library until the process exits), and it allocates nothing.
 * Limit: E * ceil(T / 8) <= 524288 (T = 16384 tokens over 256 experts
 * fits); larger requests return MOE_ERR_WORKSPACE_TOO_SMALL before anything
 * is enqueued. Out-of-range expert ids are skipped exactly as in
 * moe_dispatch (pos = -1); there is no error word to read back.
 * Every call shares the array and it keeps the last call's contents (each
 * call rewrites the tables and clears its error word first). Calls whose
 * kernels overlap on the GPU race on the array: order them on one stream.
 * The first call on each device looks up the array's device address (with
 * that device current) and keeps it for the life of the process; make that
 * first call before any stream capture. The kept address belongs to the
 * device's primary context: after cudaDeviceReset (or anything else that
 * destroys that context) it is stale, so do not call this entry point again
 * in a process that has reset the device. */
MOE_API int moe_dispatch_noalloc(const moe_config_t* cfg, const void* x,
                         const int32_t* topk_idx, int32_t* counts, int32_t* offsets,
                         int32_t* pos, int32_t* src, void* x_perm, float* x_scale,
                         void* stream);

/* ---- stage 3: grouped expert FFN -----------------------------------------
 * "L1 + Act + L2" per expert (DeepSeek V3/V4 parallel-strategy article,
 * Waved-EP section), read as one up projection, SiLU and one down projection:
 * For every expert e with rows [offsets[e], offsets[e+1]) of x_perm:
 *   h[r] = SiLU(s_r * x_perm[r] . W1[e])   (s_r = x_scale[r] with FP8, else 1)
 *   y_perm[r] = h[r] . W2[e]
 * x_perm [R, d] (dtype, or uint8 E4M3 with the FP8 payload), x_scale [R]
 * fp32 (FP8 only), offsets [E+1] int32 (non-decreasing, offsets[E] <= R;
 * rows past offsets[E] are not touched), W1 [E, d, f] and W2 [E, f, d]
 * (dtype, expert-major), h [R, f] (dtype) output, y_perm [R, d] fp32 output.
 * bf16 uses the tcgen05 tensor cores (fp32 accumulate in TMEM); fp32 uses
 * fp32 FMA. With the FP8 payload the GEMM reads the E4M3 bytes and expands
 * them to bf16 in shared memory (exact), applying s_r in its epilogue.
 * Experts with no rows read none of their weights.
 * MOE_ROUTER_SOFT_GUMBEL: x_perm is x itself, [T, d]; row r of expert e's
 * segment reads x[r - offsets[e]] (every expert reads all T rows).
 * ws: >= moe_scratch_size bytes. */
MOE_API int moe_expert_ffn(const moe_config_t* cfg, const void* x_perm,
                   const float* x_scale, const int32_t* offsets, const void* W1,
                   const void* W2, void* h, float* y_perm, void* ws,
                   size_t ws_bytes, void* stream);

/* ---- stage 4: combine ------------------------------------------------------
 * The weighted sum of a token's k expert outputs (Deepseek-MoE sync-tax
 * article, section 2.3):
 * out[t] = sum_{j=0..k-1} topk_w[t, j] * y_perm[pos[t*k + j]], accumulated in
 * fp32 in increasing j, then stored in dtype. No atomics: the result is
 * bitwise reproducible. y_perm [R, d] fp32, pos [R] int32, topk_w [T, k]
 * fp32, out [T, d] (dtype). A pos outside [0, R) contributes nothing and
 * flags MOE_ERR_BAD_INDEX. ws: >= moe_scratch_size bytes. */
MOE_API int moe_combine(const moe_config_t* cfg, const float* y_perm, const int32_t* pos,
                const float* topk_w, void* out, void* ws, size_t ws_bytes,
                void* stream);

/* ---- FP8 expert-output payload -------------------------------------------
 * The Deepseek-MoE sync-tax article (section 3.1) sends each expert output
 * vector to the combine as FP8, quantised on its own from its min and max by
 * an affine map.
 * moe_quantize_output: for each row r < R = T*k of y_perm [R, d] fp32:
 *   mn, mx = the row's min and max; zero = fp32(mx/2 + mn/2);
 *   half = fp32(mx/2 - mn/2); s = fp32(half / 448), IEEE division (1 when
 *   half = 0); y_q[r][c] = E4M3(fp32(fp32(y - zero) / s)), rounded to
 *   nearest even, saturating at +-448 (OCP E4M3, no infinities).
 *   Outputs: y_q [R, d] uint8, y_scale [R] fp32 (s), y_zero [R] fp32 (zero).
 *   No workspace; no device-side error is possible.
 * moe_combine_fp8: out[t] = sum_{j=0..k-1} topk_w[t, j] * (q * s + zero) of
 *   row pos[t*k + j], in fp32 in increasing j (each decoded value one fp32
 *   fma), stored in dtype; bitwise reproducible. A pos outside [0, R)
 *   contributes nothing and flags MOE_ERR_BAD_INDEX.
 *   ws: >= moe_scratch_size bytes (error word). */
MOE_API int moe_quantize_output(const moe_config_t* cfg, const float* y_perm, uint8_t* y_q,
                        float* y_scale, float* y_zero, void* stream);
MOE_API int moe_combine_fp8(const moe_config_t* cfg, const uint8_t* y_q, const float* y_scale,
                    const float* y_zero, const int32_t* pos, const float* topk_w,
                    void* out, void* ws, size_t ws_bytes, void* stream);

/* ---- whole layer -----------------------------------------------------------
 * Dispatch, L1 + Act + L2 and combine in sequence (DeepSeek V3/V4
 * parallel-strategy article, EP and Waved-EP sections), on one GPU:
 * moe_route -> moe_dispatch -> moe_expert_ffn -> moe_combine (or, with
 * output_fp8, moe_quantize_output -> moe_combine_fp8) on one stream, with
 * every intermediate in the workspace (>= moe_workspace_size bytes).
 * noise: as for moe_route (the soft router's Gumbel samples, else NULL).
 * No host synchronisation, so the call can be captured into a CUDA graph. */
MOE_API int moe_forward(const moe_config_t* cfg, const void* x, const void* W_g,
                const float* bias, const float* noise, const void* W1, const void* W2,
                void* out, void* ws, size_t ws_bytes, void* stream);

/* ---- whole layer for a few tokens ------------------------------------------
 * moe_forward's layer for at most MOE_FEW_MAX_TOKENS tokens (a decode step),
 * gate to combine in one kernel: the routing rules of moe_route, the experts
 * as in moe_expert_ffn, the weighted sum as in moe_combine, with every sum
 * in fp32 and h carried as two bf16 parts, so only out is rounded to bf16
 * (moe_forward rounds h too, and adds in another order). bf16 layers without
 * payloads (payload_fp8, output_fp8) or keep_z, T <= MOE_FEW_MAX_TOKENS;
 * else MOE_ERR_UNSUPPORTED. gemm_tile_n and x_perm_mode have no effect.
 * Arguments as moe_forward. ws: >= moe_forward_few_workspace_size bytes (0
 * for a configuration it refuses), 256-byte aligned, zeroed once before its
 * first use and again after a MOE_ERR_TIMEOUT; calls that share one must not
 * overlap. No atomics on values: bitwise reproducible. The kernel's blocks
 * wait on one another (a cooperative launch, one block per SM). It can be
 * captured into a graph. */
#define MOE_FEW_MAX_TOKENS 32
MOE_API size_t moe_forward_few_workspace_size(const moe_config_t* cfg);
MOE_API int moe_forward_few(const moe_config_t* cfg, const void* x, const void* W_g,
                const float* bias, const float* noise, const void* W1, const void* W2,
                void* out, void* ws, size_t ws_bytes, void* stream);

/* (No counterpart on the source pages: timing instrumentation.)
 * moe_forward that also records CUDA events (cudaEvent_t, passed as void*)
 * at the kernel boundaries, for per-kernel timing on the launching stream:
 *   events[0] before the route kernel      events[1] after route
 *   events[2] after dispatch (3 kernels; 1 with soft gating)
 *                                          events[3] = events[2] (kept for
 *   the slot; the FP8 payload is expanded  events[4] after the W1 GEMM
 *   inside the W1 GEMM)
 *   events[5] after the W2 GEMM            events[6] after the output
 *   quantisation (= events[5] without)     events[7] after combine
 * n_events must be MOE_NUM_EVENTS; any entry may be NULL (not recorded). */
#define MOE_NUM_EVENTS 8
MOE_API int moe_forward_with_events(const moe_config_t* cfg, const void* x,
                            const void* W_g, const float* bias, const float* noise,
                            const void* W1, const void* W2, void* out, void* ws,
                            size_t ws_bytes, void* const* events, int n_events,
                            void* stream);

/* (No counterpart on the source pages: inspection of intermediates.)
 * Pointers into a forward workspace, so a caller can inspect the
 * intermediates of the last moe_forward (routing, permutation, H, Y).
 * Any output pointer may be NULL. x_perm is NULL when that forward packs no
 * rows (gathered rows, soft gating). Returns MOE_ERR_INVALID_ARG for a bad
 * configuration. No device access. */
typedef struct moe_forward_views {
  int32_t* topk_idx; float* topk_w;
  int32_t* counts; int32_t* offsets; int32_t* pos; int32_t* src;
  void* x_perm; float* x_scale; void* h; float* y_perm;
  uint8_t* y_q; float* y_scale; float* y_zero;  /* NULL unless output_fp8 */
  float* z;                                     /* NULL unless keep_z */
} moe_forward_views_t;
MOE_API int moe_forward_views(const moe_config_t* cfg, void* ws, moe_forward_views_t* views);

/* ---- backward ------------------------------------------------------------
 * Gradients of a loss l through one moe_forward call, given dout = dl/dout
 * [T, d] (the output dtype): in backpropagation the gradient goes back only
 * to the activated experts (DeepSeek-V4 EP article, section 2.1), along the
 * mirror of the dispatch (Deepseek-MoE sync-tax article, section 2.4):
 *   dY[pos(t,j)] = w[t,j] dout[t]           dw[t,j] = <dout[t], Y[pos(t,j)]>
 *   dL = router Jacobian of dw (softmax over the chosen set; over the pre_k
 *        set for MOE_ROUTER_PREK_SOFTMAX; over all experts, / tau, for
 *        soft gating); no gradient flows through the choice itself
 *   dW_g = x^T dL   db = sum_t dL   dx = dL W_g^T + sum_j dX_perm[pos(t,j)]
 *   per expert e: Z = X_e W1_e (recomputed, or kept by the forward with
 *   keep_z), dW2_e = H_e^T dY_e,
 *   dZ = (dY_e W2_e^T) * SiLU'(Z), dW1_e = X_e^T dZ, dX_perm = dZ W1_e^T
 * x, W_g, bias, noise, W1, W2: the forward's inputs, unchanged. fwd_ws: the
 * workspace of that moe_forward call (>= moe_workspace_size bytes; its
 * routing, permutation, x_perm, H, Y and, with keep_z, Z are read, not
 * changed; keep_z must be the same on both calls). Outputs,
 * fp32, overwritten: dx [T, d], dW_g [d, E], dbias [E] (nullable), dW1 [E,
 * d, f], dW2 [E, f, d]; an expert with no rows gets zero gradients. ws: >=
 * moe_backward_workspace_size bytes, 256-byte aligned; its first word is
 * the backward's device error word (moe_get_device_error(ws, ...)). The
 * FP8 payloads (payload_fp8, output_fp8) have no backward:
 * MOE_ERR_UNSUPPORTED. Every tensor pointer (x, W_g, W1, W2, dout, dx,
 * dW_g, dW1, dW2) must be 16-byte aligned, else MOE_ERR_INVALID_ARG.
 * Precision: bf16 layers run the GEMMs on the tensor cores with each fp32
 * operand carried as two bf16 parts hi + lo (~2^-17 relative) against a
 * bf16 one, fp32 accumulation: dZ and dL against the weights or inputs,
 * and for dW2 either dY against H or, where 2f <= d, w H (each routed row's
 * weight times its H row) against the dout rows; dH takes the bf16 dout
 * rows themselves, the routing weight applied to the fp32 sum; fp32 layers
 * use fp32 FMA. Every sum runs in a fixed order (no atomics): the result is
 * bitwise reproducible. Asynchronous on `stream`. */
MOE_API size_t moe_backward_workspace_size(const moe_config_t* cfg);
MOE_API int moe_backward(const moe_config_t* cfg, const void* x, const void* W_g,
                 const float* bias, const float* noise, const void* W1, const void* W2,
                 const void* fwd_ws, size_t fwd_ws_bytes, const void* dout, float* dx,
                 float* dW_g, float* dbias, float* dW1, float* dW2, void* ws,
                 size_t ws_bytes, void* stream);

/* The same with a gradient of the logits from elsewhere added to the
 * router's, before it goes on to x, W_g and the bias: dlogits [T, E] fp32
 * (moe_router_loss_backward's), 4-byte aligned. */
MOE_API int moe_backward_with_dlogits(const moe_config_t* cfg, const void* x, const void* W_g,
                 const float* bias, const float* noise, const void* W1, const void* W2,
                 const void* fwd_ws, size_t fwd_ws_bytes, const void* dout,
                 const float* dlogits, float* dx, float* dW_g, float* dbias, float* dW1,
                 float* dW2, void* ws, size_t ws_bytes, void* stream);

/* ---- norms around a block -----------------------------------------------
 * (No counterpart on the source pages: the expert layer's neighbours in a
 * transformer block.) Root-mean-square norms before and after a block, fused
 * with the block's gate and the residual scale. With rstd(v) = 1 /
 * sqrt(mean(v^2) + eps) over a row's d values, b the block's output:
 *   out = alpha x + beta g * (b rstd(b) w_post)    (post half)
 *   n   = out rstd(out) w_pre                      (pre half: the next
 *                                                   block's input)
 * Either half may be left out: b = NULL leaves out the post half (out is x;
 * alpha, beta and the gate are not used), w_pre = NULL the pre half. n is
 * taken from the fp32 out, before its rounding; sums are fp32. A finite row
 * whose sum of squares passes the fp32 range has rstd 0: its norm, and what
 * comes back through it, is 0. */
enum {
  MOE_GATE_NONE = 0,    /* g = 1 */
  MOE_GATE_TOKEN = 1,   /* gate [T] fp32 */
  MOE_GATE_CHANNEL = 2, /* gate [d] fp32 */
  MOE_GATE_ELEMENT = 3  /* gate [T, d] (dtype) */
};

typedef struct moe_norm_config {
  int32_t T;     /* rows, >= 0 */
  int32_t d;     /* row length, multiple of 64, at most 65536 */
  int32_t dtype; /* MOE_DTYPE_*: x, b, out, n, dout, dx, db, an element gate */
  int32_t gate;  /* MOE_GATE_* */
  float eps;     /* finite, > 0 */
  float alpha;   /* residual scale, finite */
  float beta;    /* branch scale, finite */
} moe_norm_config_t;

/* x, b [T, d]; w_post, w_pre [d] fp32; gate as cfg->gate says. Outputs:
 * out [T, d] (NULL without the post half), n [T, d] (NULL without the pre
 * half), rstd_post, rstd_pre [T] fp32 (what the backward reads; nullable).
 * Outputs may not overlap inputs or one another (MOE_ERR_INVALID_ARG; the
 * backward's likewise). Every tensor pointer but the [T] ones is 16-byte
 * aligned. */
MOE_API int moe_block_norm(const moe_norm_config_t* cfg, const void* x, const void* b,
                   const float* w_post, const void* gate, const float* w_pre, void* out,
                   void* n, float* rstd_post, float* rstd_pre, void* stream);

/* Gradients of moe_block_norm's inputs, given dout [T, d] (the gradient that
 * reaches out by other ways than n: the next residual's) and dn [T, d] fp32
 * (moe_backward's dx; NULL without the pre half). x, b, weights and gate: the
 * forward's, unchanged; rstd_*: what it wrote. out is formed again from x and
 * b, in fp32 (its rounding does not reach the gradients); x is not read
 * without the pre half and may be NULL there.
 * Outputs, overwritten: dx [T, d] (of x, through the residual), db [T, d],
 * dw_post, dw_pre [d] fp32, dgate (gate's shape; fp32, or dtype for an
 * element gate); those of a half left out, and dgate without a gate, are
 * NULL. ws: >= moe_block_norm_backward_workspace_size bytes (0 for an
 * invalid configuration), 256-byte aligned; no zeroing. Two kernels, no
 * atomics: bitwise reproducible. T = 0 zeroes the weights' gradients; the
 * tensors of T rows, empty then, may be NULL. */
MOE_API size_t moe_block_norm_backward_workspace_size(const moe_norm_config_t* cfg);
MOE_API int moe_block_norm_backward(const moe_norm_config_t* cfg, const void* dout,
                   const float* dn, const void* x, const void* b, const float* w_post,
                   const void* gate, const float* w_pre, const float* rstd_post,
                   const float* rstd_pre, void* dx, void* db, float* dw_post, void* dgate,
                   float* dw_pre, void* ws, size_t ws_bytes, void* stream);

/* ---- microscaled 4-bit expert products --------------------------------------
 * (No counterpart on the source pages, whose payloads stop at 8 bits.) The
 * expert products of moe_expert_ffn with both operands in 4 bits: OCP
 * microscaling, MXFP4. Blocks of 32 values along the contraction share one
 * power-of-two scale, a byte s (E8M0: 2^(s - 127)); each value is E2M1:
 *   s - 127 = max(floor(log2(amax)) - 2, -127); s = 127 for a block of zeros,
 *   255 (which stands for NaN) for a block with an infinity or a NaN;
 *   code = E2M1(v / 2^(s - 127)), to nearest even, saturating at +-6.
 * Codes lie two to a byte, the even k in the low half: rows [R, K / 2],
 * weights [E, N, K / 2] (transposed: k innermost). Scales lie as the tensor
 * cores read them, in chunks of 128 rows (or columns n) x 4 blocks, 512
 * bytes: row i, block j at (i % 32) * 16 + (i / 32) * 4 + j. Weights:
 * [E][ceil(N / 128)][ceil(K / 128)] chunks. Rows: [tile][ceil(K / 128)]
 * chunks, where the tiles are each expert's segment cut into 128 rows, one
 * expert after the other, so they go with the offsets they were made for.
 * Every code and scale pointer is 16-byte aligned. */
typedef struct moe_mx4_config {
  int32_t R;         /* routed rows, 0..2^24 */
  int32_t K;         /* contraction, multiple of 64, at most 65536 */
  int32_t N;         /* output features, multiple of 64, at most 65536 */
  int32_t E;         /* experts, 1..256 (1: a plain linear layer, offsets {0, R}) */
  int32_t dtype;     /* MOE_DTYPE_*: x, W and what the dequantisers write */
  int32_t out_dtype; /* MOE_DTYPE_*: the product's output */
  int32_t silu;      /* 1: the product ends in SiLU (the W1 pass); else 0 */
  int32_t x_rows;    /* rows of x where quantised rows are gathered, >= 0 */
} moe_mx4_config_t;

/* Sizes in bytes (0 for an invalid configuration): the rows' scales, the
 * weights' scales, and the workspace of the two calls that take one (an
 * error word and the product's split sums; 256-byte aligned; zero it once
 * before its first use and again after a MOE_ERR_TIMEOUT; calls that share
 * one must not overlap). */
MOE_API size_t moe_mx4_row_scale_size(const moe_mx4_config_t* cfg);
MOE_API size_t moe_mx4_weight_scale_size(const moe_mx4_config_t* cfg);
MOE_API size_t moe_mx4_workspace_size(const moe_mx4_config_t* cfg);

/* Expert weights W [E, K, N] (dtype) -> wq [E, N, K / 2], w_scale; done once
 * where the weights are loaded. */
MOE_API int moe_mx4_quantize_weights(const moe_mx4_config_t* cfg, const void* W, uint8_t* wq,
                   uint8_t* w_scale, void* stream);

/* Rows of x (dtype) -> q [R, K / 2], scale: row r of the layout is x[r], or
 * x[src[r]] with src (the dispatch's; x then has x_rows rows), so the packed
 * bf16 rows need not exist. Rows outside [offsets[0], offsets[E]) are not
 * touched. A src outside [0, x_rows) gives a row of zeros, offsets that fall
 * or leave [0, R] give nothing, and both flag MOE_ERR_BAD_INDEX. */
MOE_API int moe_mx4_quantize_rows(const moe_mx4_config_t* cfg, const void* x,
                   const int32_t* src, const int32_t* offsets, uint8_t* q, uint8_t* scale,
                   void* ws, size_t ws_bytes, void* stream);

/* out[r] = q[r] . wq[e] (fp32 sums, then SiLU with cfg->silu, then rounded
 * to out_dtype) for the rows r of each expert e's segment [offsets[e],
 * offsets[e + 1]); out [R, N]. Offsets that fall or leave [0, R] write
 * nothing and flag MOE_ERR_BAD_INDEX. Bitwise reproducible. */
MOE_API int moe_mx4_product(const moe_mx4_config_t* cfg, const uint8_t* q, const uint8_t* scale,
                   const uint8_t* wq, const uint8_t* w_scale, const int32_t* offsets,
                   void* out, void* ws, size_t ws_bytes, void* stream);

/* The values codes and scales stand for (exact in both types): W [E, K, N],
 * rows [R, K]. Offsets that fall or leave [0, R] write no rows (and, these calls
 * having no workspace, flag nothing: moe_mx4_quantize_rows did). */
MOE_API int moe_mx4_dequantize_weights(const moe_mx4_config_t* cfg, const uint8_t* wq,
                   const uint8_t* w_scale, void* W, void* stream);
MOE_API int moe_mx4_dequantize_rows(const moe_mx4_config_t* cfg, const uint8_t* q,
                   const uint8_t* scale, const int32_t* offsets, void* x, void* stream);

/* ---- 8-bit expert products, forward and backward ------------------------------
 * (The source pages quantise what is exchanged; here both sides of the
 * products are, and of their gradients.) E4M3 codes (largest 448) with one
 * power-of-two scale, a byte s, for each block of 128:
 *   s - 127 = the least e >= -127 with amax <= 448 2^e; s = 127 for a block
 *   of zeros, 255 (which stands for NaN) for one with an infinity or a NaN;
 *   code = E4M3(v / 2^(s - 127)), to nearest even (nothing saturates).
 * Rows: blocks of 128 along a row; codes [R, C], scales [R, pitch] bytes,
 * pitch = ceil(C / 128) rounded up to 4 (the padding is not read). Columns:
 * blocks of 128 rows of one expert, whose segment is cut into tiles of 128
 * from its start, one expert after the other; codes [tile * 128 + row, C],
 * zeros past a segment's end, scales [tile, ceil(C / 128), 128], those of 128
 * columns in the order the tensor core reads them: column i at (i % 32) * 4 +
 * i / 32 (127 past C). Weights: blocks of 128 x 128
 * of each W[e]; codes [E, K, N] as W lies, scales [E, ceil(K / 128),
 * ceil(N / 128)]: the one copy serves the product and its transpose. C is K
 * (rows of x) or N (rows of dy). Code pointers are 16-byte aligned, the
 * scales of rows and columns, src, row_weight and offsets 4-byte. */
typedef struct moe_fp8_config {
  int32_t R;         /* routed rows, 0..2^24 */
  int32_t K;         /* W's rows (the product's contraction), multiple of 64, at most 65536 */
  int32_t N;         /* W's columns, multiple of 64, at most 65536 */
  int32_t E;         /* experts, 1..256 (1: a plain linear layer, offsets {0, R}) */
  int32_t dtype;     /* MOE_DTYPE_*: x, z, W and what the dequantisers write */
  int32_t out_dtype; /* MOE_DTYPE_*: the products' output (weight gradients are fp32) */
  int32_t silu;      /* 1: the product ends in SiLU (the W1 pass); else 0 */
  int32_t x_rows;    /* rows of x where quantised rows are gathered, >= 0 */
} moe_fp8_config_t;

/* What is quantised, x or a function of it */
enum {
  MOE_ACT_NONE = 0,      /* x */
  MOE_ACT_SILU = 1,      /* SiLU(x): the rows of the second product from the
                          * first one's pre-activation */
  MOE_ACT_SILU_GRAD = 2  /* x SiLU'(z): what goes back past the activation */
};

/* Sizes (0 for an invalid configuration): bytes of the scales of rows of
 * `cols` columns; rows of a columns' code tensor (a multiple of 128; a
 * 128th of them are tiles); bytes of the weights' scales; bytes of the
 * workspace (an error word and split sums; 256-byte aligned; zero it once
 * before its first use and again after a MOE_ERR_TIMEOUT; calls that share
 * one must not overlap). */
MOE_API size_t moe_fp8_row_scale_size(const moe_fp8_config_t* cfg, int32_t cols);
MOE_API size_t moe_fp8_column_rows(const moe_fp8_config_t* cfg);
MOE_API size_t moe_fp8_weight_scale_size(const moe_fp8_config_t* cfg);
MOE_API size_t moe_fp8_workspace_size(const moe_fp8_config_t* cfg);

/* Expert weights W [E, K, N] (dtype) -> wq, w_scale. */
MOE_API int moe_fp8_quantize_weights(const moe_fp8_config_t* cfg, const void* W, uint8_t* wq,
                   uint8_t* w_scale, void* stream);

/* Rows of x (dtype, `cols` = K or N columns) -> rows (q, scale), columns (cq,
 * cscale) or both in one pass; the form left out is NULL. Row r of the
 * layout is x[r], or x[src[r]] with src (x then has x_rows rows), times
 * row_weight[r] (fp32 [R]; NULL: 1) and through `act` (MOE_ACT_*; z [R, cols]
 * with MOE_ACT_SILU_GRAD, else NULL), all in fp32. Rows outside [offsets[0],
 * offsets[E]) are not touched. A src outside [0, x_rows) gives a row of zeros,
 * offsets that fall or leave [0, R] give nothing, and both flag
 * MOE_ERR_BAD_INDEX. Outputs may not overlap inputs or one another
 * (MOE_ERR_INVALID_ARG, as in every call here). */
MOE_API int moe_fp8_quantize_rows(const moe_fp8_config_t* cfg, int32_t cols, const void* x,
                   const int32_t* src, const float* row_weight, int32_t act, const void* z,
                   const int32_t* offsets, uint8_t* q, uint8_t* scale, uint8_t* cq,
                   uint8_t* cscale, void* ws, size_t ws_bytes, void* stream);

/* transposed 0: out[r] = rows q[r] . wq[e], q of K columns, out [R, N] (then
 * SiLU with cfg->silu); 1: out[r] = q[r] . wq[e]^T, q of N columns, out [R, K]
 * (the gradient of the product's rows; cfg->silu must be 0:
 * MOE_ERR_UNSUPPORTED), for the rows of each expert e's segment. fp32 sums,
 * rounded to out_dtype. The tensor cores' additions drop what is below the last
 * place: up to 128 of them in a row where out_dtype is fp32 (64 for weight
 * gradients; the whole contraction where it is bf16), the parts then added to
 * nearest. Of random values, the norm of an fp32 result's error stays below 64
 * (32) half steps of fp32 of the result's, typically 4. Offsets that fall or
 * leave [0, R] write nothing and flag MOE_ERR_BAD_INDEX; rows of no segment are
 * not written. Bitwise reproducible. */
MOE_API int moe_fp8_product(const moe_fp8_config_t* cfg, int32_t transposed, const uint8_t* q,
                   const uint8_t* scale, const uint8_t* wq, const uint8_t* w_scale,
                   const int32_t* offsets, void* out, void* ws, size_t ws_bytes,
                   void* stream);

/* dW[e] = sum over expert e's rows of x[r]^T dy[r], fp32 [E, K, N], from the
 * columns of x and of dy made for the same offsets; zeros for an expert
 * without rows. Bad offsets as above. Bitwise reproducible. */
MOE_API int moe_fp8_weight_grad(const moe_fp8_config_t* cfg, const uint8_t* xq,
                   const uint8_t* x_scale, const uint8_t* dyq, const uint8_t* dy_scale,
                   const int32_t* offsets, float* dW, void* ws, size_t ws_bytes, void* stream);

/* The values codes and scales stand for (exact in both types but for bf16's
 * subnormal numbers): W [E, K, N], rows [R, cols]. */
MOE_API int moe_fp8_dequantize_weights(const moe_fp8_config_t* cfg, const uint8_t* wq,
                   const uint8_t* w_scale, void* W, void* stream);
MOE_API int moe_fp8_dequantize_rows(const moe_fp8_config_t* cfg, int32_t cols, const uint8_t* q,
                   const uint8_t* scale, void* x, void* stream);

/* ---- the router's losses -----------------------------------------------------
 * (No counterpart on the source pages, which measure the experts' load and
 * leave its training to others.) Over the tokens t of sequence s that count
 * (n_s of them, of which c_se chose expert e):
 *   p_t = softmax(L_t)  f_se = E c_se / (k n_s)  P_se = sum_t p_te / n_s
 *   balance = sum_s sum_e f_se P_se / S'    over the S' sequences with n_s > 0
 *   z       = sum_t lse_t^2 / N             lse_t = log sum_e exp(L_te)
 *   loss    = cfg->balance * balance + cfg->z * z
 * One sequence (S = 1) makes it the loss of the batch. The counts are
 * constants to the gradient. */
typedef struct moe_router_loss_config {
  int32_t T;     /* tokens, 0..2^26 */
  int32_t E;     /* experts, 1..256 */
  int32_t k;     /* experts per token, 1..min(E, 16) */
  int32_t S;     /* sequences, 1..2^20 */
  float balance; /* coefficients, finite */
  float z;
} moe_router_loss_config_t;

/* Workspace bytes (0 for an invalid configuration); 256-byte aligned; zero it
 * once before its first use; calls that share one must not overlap. */
MOE_API size_t moe_router_loss_workspace_size(const moe_router_loss_config_t* cfg);

/* logits [T, E] fp32 and topk_idx [T, k] as moe_route gives them. seq_offsets
 * [S + 1]: sequence s is the tokens [seq_offsets[s], seq_offsets[s + 1]); NULL
 * (S = 1 only): all T. mask [T] bytes, 0 for a token that does not count;
 * NULL: all do. Tokens of no sequence do not count, and neither their logits
 * nor those of masked tokens are read.
 * Outputs: loss [3] (the loss, balance, z; 0 with no token), counts [S, E]
 * (c), tokens [S + 2] (n_s, then S' and N), lse [T] (0 where masked; not
 * written for tokens of no sequence). Logits of -infinity are experts that a
 * token may not take (p = 0); a token with nothing else, a +infinity or a NaN
 * has no softmax: the losses are NaN, and so is its own gradient, unless it is
 * masked. Offsets that fall or leave [0, T] write nothing but values of lse,
 * an expert id outside [0, E) is not counted, and both flag
 * MOE_ERR_BAD_INDEX. Bitwise reproducible. */
MOE_API int moe_router_loss(const moe_router_loss_config_t* cfg, const float* logits,
                   const int32_t* topk_idx, const int32_t* seq_offsets, const uint8_t* mask,
                   float* loss, int32_t* counts, int32_t* tokens, float* lse, void* ws,
                   size_t ws_bytes, void* stream);

/* dlogits [T, E] fp32 = dloss * the gradient of loss[0] (dloss: one fp32 on the
 * device; NULL: 1), 0 for tokens that do not count. logits, seq_offsets, mask:
 * the forward's; counts, tokens, lse: what it wrote. */
MOE_API int moe_router_loss_backward(const moe_router_loss_config_t* cfg, const float* logits,
                   const int32_t* seq_offsets, const uint8_t* mask, const int32_t* counts,
                   const int32_t* tokens, const float* lse, const float* dloss,
                   float* dlogits, void* stream);

/* ---- dropout of a block's branch ---------------------------------------------
 * (No counterpart on the source pages: the block around the layer.)
 *   out = residual + keep x / (1 - p')     dx = keep dout / (1 - p')
 * The mask is drawn again wherever it is needed and never stored: element i
 * (of T d) takes 16 bits of Philox 4x32 with ten rounds (Salmon et al., SC
 * 2011), counter (i / 8 low, i / 8 high, site, step), key the 64-bit seed, word
 * (i % 8) / 2, its low half for an even i; it is kept where those bits are at
 * least thr = min(round(65536 p), 65535), and p' = thr / 65536. */
typedef struct moe_dropout_config {
  int32_t T;     /* rows, 0..2^24 */
  int32_t d;     /* row length, multiple of 64, at most 65536 */
  int32_t dtype; /* MOE_DTYPE_*: x, residual, out, dout, dx */
  int32_t site;  /* which of a model's dropouts this is, >= 0 */
  float p;       /* share that is dropped, 0 <= p < 1 */
} moe_dropout_config_t;

/* state: two int64 in device memory, the seed and the step (its low 32 bits
 * are used), read by the kernel, so that a captured graph draws anew when
 * they change; 8-byte aligned. residual may be NULL (none). out may be x or
 * residual itself; other overlaps are MOE_ERR_INVALID_ARG. A dropped element
 * is the residual alone, whatever x holds there. The residual's gradient is
 * dout. The backward takes the forward's config and state. */
MOE_API int moe_dropout(const moe_dropout_config_t* cfg, const void* x, const void* residual,
                   const int64_t* state, void* out, void* stream);
MOE_API int moe_dropout_backward(const moe_dropout_config_t* cfg, const void* dout,
                   const int64_t* state, void* dx, void* stream);

/* ---- errors --------------------------------------------------------------
 * moe_get_device_error synchronises `stream`, reads the workspace error
 * word, clears it, and returns MOE_OK, MOE_ERR_BAD_INDEX or MOE_ERR_TIMEOUT
 * (or MOE_ERR_LAUNCH if the stream itself reports an error).
 * moe_clear_device_error enqueues a clear of the error word on `stream`. */
MOE_API int moe_get_device_error(void* ws, void* stream);
MOE_API int moe_clear_device_error(void* ws, void* stream);
MOE_API const char* moe_strerror(int status);

/* Number of kernels one moe_forward call launches for cfg (0 if invalid). */
MOE_API int moe_forward_kernel_count(const moe_config_t* cfg);

/* ---- test hook: the bounded-wait path ---------------------------------------
 * Every wait inside the library's kernels gives up after a bound (2 s by
 * default: a wait that long means the GPU is not making progress), flags
 * MOE_ERR_TIMEOUT in the workspace's error word and lets the kernel finish
 * cleanly (copies and tensor-core work in flight are awaited, tensor memory
 * is freed), so the context stays usable. This call sets, for launches made
 * after it in this process, the bound of one of those waits in the grouped
 * expert GEMM: its epilogue's wait for a finished accumulator, the one a
 * test can make run out without a copy being left in flight (a tiny bound
 * such as 1 ns does it). The GEMM then reports MOE_ERR_TIMEOUT, having taken
 * up to the default bound to wind down. 0 restores the default. Not for use
 * outside tests: the library itself never shortens a bound. Returns
 * MOE_OK. */
MOE_API int moe_set_gemm_epilogue_wait_ns(uint64_t ns);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_MOE_H_ */
