/*
 * moe.h -- C ABI of the routed-expert MoE layer on MI355X (gfx950).
 *
 * The layer (pages: "kimi-k3-in-c", section 4 "Reduction one: the experts
 * already ship at half a byte", section 9 "Picking 16 experts of 896" and
 * "Three invariants"; "Part 4 - Lecture 01", section 1 model table):
 *
 *   route:   logit[t][e] = sum_i x[t][i] * Wr[e][i];  s = sigmoid(logit);
 *            pick the k experts with the largest s + bias (ties -> lower id);
 *            weight_j = s[id_j] / sum_j s[id_j] (if renorm) * routed_scale.
 *            The bias steers selection only; weights use the unbiased s.
 *   experts: for each chosen expert e: g = W1_e x, u = W3_e x, h = act(g, u),
 *            y = W2_e h, with W1, W3, W2 in MXFP4 (E2M1 code per weight,
 *            E8M0 scale byte per 32 consecutive weights of a row).
 *   combine: out[t] = sum_j weight_j * y_j + sum_s FFN_shared_s(x[t]), the
 *            shared experts bf16, on the same x, added unweighted.
 *   act:     SiTU-GLU  h = b1*tanh(g/b1)*sigmoid(g) * b2*tanh(u/b2)
 *            (sigmoid of the uncapped g; K3 uses b1 = 4, b2 = 25), or
 *            SwiGLU    h = g*sigmoid(g)*u.
 *
 * Conventions (every call):
 *  - All pointers are DEVICE pointers owned by the caller; the library
 *    allocates nothing, keeps no state of its own between calls (apart from
 *    the one setting of moe_set_one_token_router_wait) and never
 *    synchronises the host.  Work is enqueued on `stream` (a hipStream_t; NULL = the null
 *    stream) and may be captured into a HIP graph (no memset, no allocation).
 *  - Arguments are validated before anything is launched; on any error
 *    nothing is enqueued and a negative moe_status is returned.
 *  - T = 0 is a valid no-op.
 *  - Calls that share a workspace must not overlap in time.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_EINVAL = -1,        /* a null/misaligned pointer, a bad size or enum      */
    MOE_EUNSUPPORTED = -2,  /* valid but outside the supported shape range below  */
    MOE_EWORKSPACE = -3,    /* ws_bytes < moe_workspace_bytes(desc, T)            */
    MOE_EHIP = -4           /* a HIP launch failed (hipGetLastError != success)   */
} moe_status;

typedef enum { MOE_ACT_SITU = 0, MOE_ACT_SWIGLU = 1 } moe_act;

/* which outputs moe_expert_forward / moe_layer write */
typedef enum { MOE_OUT_BF16 = 0, MOE_OUT_F32 = 1, MOE_OUT_BOTH = 2 } moe_out_mode;

/* which expert kernels run: AUTO picks the dequant-fused GEMV for up to 12
 * tokens and the grouped MFMA GEMM above (moe_path_for reports it); one
 * token on the GEMV path takes fused one-token kernels where their limits
 * allow (SiTU with b1*b2 <= 65504 among them).
 * The MFMA path needs d and F to be multiples of 256, every activation
 * operand below 2 GiB (T*k*F, T*d and T*S*F two-byte values) and, under
 * SiTU, b1*b2 <= 65504; AUTO falls back to GEMV outside that range, and an
 * explicit MOE_PATH_MFMA call returns MOE_EUNSUPPORTED.
 *
 * Precision of the activation H = act(g, u) between the gate/up and the down
 * products: the GEMV path keeps it in fp32; the one-token kernels and the
 * MFMA path store it in fp16 (relative rounding 2^-11), the MFMA path's
 * shared experts included: their down product takes the bf16 weights as
 * fp16 (exact in [2^-17, 65504]; smaller ones off by at most 2^-25; a pass
 * that meets a larger one is computed again exactly).  SiTU bounds |h| by
 * b1*b2, which is why those two paths need b1*b2 <= 65504 (the largest
 * fp16).  SwiGLU is unbounded: the one-token kernels never take it, and on
 * the MFMA path an |h| above 65504 becomes inf in H, so that token's outputs
 * come out inf or NaN (never a finite wrong value); MOE_PATH_GEMV keeps such
 * layers finite at any T. */
typedef enum { MOE_PATH_AUTO = 0, MOE_PATH_GEMV = 1, MOE_PATH_MFMA = 2 } moe_path;

/*
 * One layer.  Every field is required (there are no defaults).
 * Shapes: E = n_experts, k = top_k, d = d_model, F = d_ffn, S = n_shared.
 * Supported: 1 <= k <= E <= 1024, k <= 64, d and F multiples of 32 in
 * [32, 4096], 0 <= S <= 8; otherwise MOE_EUNSUPPORTED.
 *
 * MXFP4 tensors are in the checkpoint layout, row-major per expert: codes
 * [E][rows][cols/2] bytes, the low nibble of byte c/2 holding column c when c
 * is even and the high nibble column c+1; scales [E][rows][cols/32] E8M0 bytes
 * (value 2^(b-127); byte 255 makes its 32 weights contribute zero).
 * W1 (gate) and W3 (up) are [F rows][d cols]; W2 (down) is [d rows][F cols].
 * Code arrays must be 16-byte aligned; scale arrays need no alignment.
 */
typedef struct {
    int32_t n_experts, top_k, d_model, d_ffn, n_shared;
    int32_t renorm;          /* 1: weights renormalised to sum to 1 (K3: 1)      */
    float routed_scale;      /* multiplies every routed weight (K3: 1.0)         */
    int32_t act;             /* moe_act                                         */
    float situ_b1, situ_b2;  /* SiTU betas (K3: 4.0, 25.0); unused for SwiGLU     */
    int32_t path;            /* moe_path                                        */
    const float *router_w;   /* [E][d] fp32, 16-byte aligned                     */
    const float *router_bias;/* [E] fp32 selection bias, or NULL for none        */
    const uint8_t *w1_q, *w1_s;  /* gate: [E][F][d/2], [E][F][d/32]             */
    const uint8_t *w3_q, *w3_s;  /* up:   [E][F][d/2], [E][F][d/32]             */
    const uint8_t *w2_q, *w2_s;  /* down: [E][d][F/2], [E][d][F/32]             */
    const uint16_t *sh_w1;   /* shared gate [S][F][d] bf16 bits, 16-byte aligned  */
    const uint16_t *sh_w3;   /* shared up   [S][F][d] bf16                        */
    const uint16_t *sh_w2;   /* shared down [S][d][F] bf16                        */
} moe_layer_desc;

/* Workspace bytes a call with up to max_tokens tokens needs (0 if the
 * descriptor is invalid or unsupported).  Pass a buffer of at least this
 * size, 256-byte aligned, to the calls below.  Its contents need no
 * initialisation and carry nothing a caller reads.  (The one-token kernel
 * hands the router logits, and the signals that a block's activations are
 * stored, between its blocks through slots at the start of the workspace,
 * each tagged with the call's epoch, a counter kept there that every call
 * advances; a slot counts only with the running call's tag.  Slots earlier
 * calls left never carry it, and other contents carry it only by a
 * coincidence of 1 in 2^32 per slot, so the workspace may start with any
 * bytes.) */
size_t moe_workspace_bytes(const moe_layer_desc *desc, int32_t max_tokens);

/* The expert path (MOE_PATH_GEMV or MOE_PATH_MFMA) a call with T tokens
 * takes; a negative moe_status if desc is invalid. */
int32_t moe_path_for(const moe_layer_desc *desc, int32_t T);

/*
 * Router only.  x: [T][d] bf16 bits (16-byte aligned).
 * ids: [T][k] int32 -- each token's experts in descending selection score
 *      (s + bias), ties to the lower id.
 * weights: [T][k] fp32 -- the routing weights of those experts, same order.
 * counts: [E] int32 or NULL -- counts[e] = number of tokens that picked e.
 */
moe_status moe_route(const moe_layer_desc *desc, const uint16_t *x, int32_t T,
                     int32_t *ids, float *weights, int32_t *counts,
                     void *ws, size_t ws_bytes, void *stream);

/*
 * Experts for a given routing (ids/weights as moe_route writes them).
 * An id outside [0, E) drops that term.  An id given more than once in a
 * token's row (moe_route never does that) adds each of its terms: the layer
 * runs that expert once for the token, with the weights of its slots summed
 * in slot order, since w1*FFN_e(x) + w2*FFN_e(x) = (w1 + w2)*FFN_e(x).
 * include_shared: 1 adds the shared experts, 0 leaves them out.
 * out_mode picks the outputs: out_bf16 [T][d] bf16 bits (round to nearest
 * even of the fp32 result) and/or out_f32 [T][d] fp32; the one not asked
 * for may be NULL.  moe_route followed by moe_expert_forward(include_shared
 * = 1) gives bit-for-bit the results of moe_layer.
 */
moe_status moe_expert_forward(const moe_layer_desc *desc, const uint16_t *x, int32_t T,
                              const int32_t *ids, const float *weights,
                              int32_t include_shared, uint16_t *out_bf16, float *out_f32,
                              int32_t out_mode, void *ws, size_t ws_bytes, void *stream);

/*
 * Whole layer: route, experts, shared experts, combine.  ids_opt/weights_opt
 * ([T][k]) and counts_opt ([E]) receive the routing when non-NULL.
 */
moe_status moe_layer(const moe_layer_desc *desc, const uint16_t *x, int32_t T,
                     uint16_t *out_bf16, float *out_f32, int32_t out_mode,
                     int32_t *ids_opt, float *weights_opt, int32_t *counts_opt,
                     void *ws, size_t ws_bytes, void *stream);

/*
 * moe_layer without a caller workspace, for callers that cannot allocate or
 * hold one (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc).  Arguments and results are those of moe_layer, bit for
 * bit; the call allocates nothing (no hipMalloc, no allocating library
 * routine).  Its workspace is a static device array of MOE_NOALLOC_WS_BYTES
 * inside the library, one per GPU, held until the process ends and shared
 * by every moe_layer_noalloc call on that GPU: calls that overlap in time
 * on one GPU (two streams, two threads) race on it and must not be issued.
 * A call that would need more (moe_workspace_bytes(desc, T) above
 * MOE_NOALLOC_WS_BYTES; at the Kimi-K3 shape about 170 tokens) returns
 * MOE_EWORKSPACE before anything is launched.  The array needs no
 * initialisation and keeps the last call's contents, which carry nothing a
 * caller reads.
 */
#define MOE_NOALLOC_WS_BYTES ((size_t)128 << 20)
moe_status moe_layer_noalloc(const moe_layer_desc *desc, const uint16_t *x, int32_t T,
                             uint16_t *out_bf16, float *out_f32, int32_t out_mode,
                             int32_t *ids_opt, float *weights_opt, int32_t *counts_opt,
                             void *stream);

/*
 * moe_layer with phase timing: records the caller's HIP events (hipEvent_t
 * handles, exactly MOE_TIMED_EVENTS of them) on `stream` at the phase
 * boundaries: events[0] before the router, [1] after the router logits (and,
 * on the GEMV path, the shared experts' gate/up, which share that launch),
 * [2] after top-k and dispatch, [3] after the expert gate/up kernel (with the
 * activation; on the GEMV path also the shared experts' down), [4] after the
 * expert down kernel, [5] after the combine.  hipEventElapsedTime of consecutive events
 * gives each phase's device time.  Results equal moe_layer's bit for bit.
 */
#define MOE_TIMED_EVENTS 6
moe_status moe_layer_timed(const moe_layer_desc *desc, const uint16_t *x, int32_t T,
                           uint16_t *out_bf16, float *out_f32, int32_t out_mode,
                           void *ws, size_t ws_bytes, void *stream, void *const *events);

/* The one-token kernel's hand-offs between its blocks: a block that has
 * waited this many microseconds (default 50) for router logits other blocks
 * compute, or four times as long for another block's stored activations,
 * computes the missing ones itself, the same sums, so the same bits; no wait
 * depends on another block being resident.  Process-wide; it applies to
 * calls enqueued after it returns (a captured graph keeps the value it was
 * captured with).  MOE_EINVAL for a negative value. */
moe_status moe_set_one_token_router_wait(int32_t microseconds);

/*
 * Kimi-K3's Stable LatentMoE around the routed experts ("kimi-k3-in-c",
 * section 9, k3_moe, its six steps; section 5, k3_rmsnorm; section 2, the
 * K3Cfg fields latent, latent_norm and rms_eps):
 *
 *   1. route on the FULL-width x[t] (hidden wide), as moe_route does;
 *   2. z = W_down x[t]                    (W_down [latent][hidden] bf16);
 *   3. a = sum_j weight_j * FFN_{id_j}(z) (the routed experts, in the latent);
 *   4. n = RMSNorm(a) * norm_w            (of the AGGREGATE, not per expert:
 *                                          n_i = a_i * inv * w_i with
 *                                          inv = 1 / sqrt(sum a^2 / latent
 *                                          + rms_eps), if latent_norm);
 *   5. out = W_up n                       (W_up [hidden][latent] bf16);
 *   6. out += sum_s FFN_shared_s(x[t])    (full width, on the ORIGINAL x,
 *                                          added unweighted).
 *
 * Shapes: E, k, F, S as for moe_layer_desc; H = hidden, L = latent.
 * Supported: H a multiple of 32 in [32, 8192], L one in [32, 4096],
 * L + S*F <= 16384 and the moe_layer_desc limits on E, k, F and S;
 * otherwise MOE_EUNSUPPORTED.  The MFMA path (AUTO above 3 tokens) also needs H and
 * L multiples of 256 and the moe_layer_desc MFMA limits; AUTO falls back to
 * GEMV outside them.
 *
 * Precision: the latent z reaches the MXFP4 experts as fp16 with one
 * power-of-two scale per token (11 significant bits); the normed aggregate
 * reaches W_up in fp32 (GEMV) or in fp16 (MFMA, W_up taken as fp16; a pass
 * whose sums come out non-finite, an element past fp16's range, is computed
 * again on two bf16 parts, 16 bits); every product accumulates in fp32, sums
 * of squares in double.  The experts' H is as for moe_layer: fp32 on the GEMV
 * path; fp16 on the MFMA path and at one token on the GEMV path, whose
 * routed experts then run in the one-token kernel (L a multiple of 512,
 * SiTU with b1*b2 <= 65504).
 *
 * The expert tensors are those of moe_layer_desc with d = latent (W1, W3
 * [E][F][L/2] + [E][F][L/32]; W2 [E][L][F/2] + [E][L][F/32]); router and
 * shared experts take the hidden width.  Alignment: code arrays, router_w,
 * down, up and the shared weights 16 bytes.
 */
typedef struct {
    int32_t n_experts, top_k, hidden, latent, d_ffn, n_shared;
    int32_t renorm;          /* as in moe_layer_desc (K3: 1)                     */
    float routed_scale;      /* (K3: 1.0)                                        */
    int32_t act;             /* moe_act                                         */
    float situ_b1, situ_b2;  /* (K3: 4.0, 25.0)                                  */
    int32_t latent_norm;     /* 1: RMSNorm of the aggregate (K3: 1); 0: none     */
    float rms_eps;           /* inside the square root (K3: 1e-5), >= 0           */
    int32_t path;            /* moe_path                                        */
    const float *router_w;   /* [E][H] fp32                                      */
    const float *router_bias;/* [E] fp32 selection bias, or NULL                 */
    const uint16_t *down;    /* [L][H] bf16 bits                                 */
    const uint8_t *w1_q, *w1_s;  /* gate: [E][F][L/2], [E][F][L/32]             */
    const uint8_t *w3_q, *w3_s;  /* up:   [E][F][L/2], [E][F][L/32]             */
    const uint8_t *w2_q, *w2_s;  /* down: [E][L][F/2], [E][L][F/32]             */
    const float *norm_w;     /* [L] fp32 RMSNorm weight, or NULL for weight 1     */
    const uint16_t *up;      /* [H][L] bf16 bits                                 */
    const uint16_t *sh_w1;   /* shared gate [S][F][H] bf16                        */
    const uint16_t *sh_w3;   /* shared up   [S][F][H] bf16                        */
    const uint16_t *sh_w2;   /* shared down [S][H][F] bf16                        */
} moe_latent_desc;

/* Workspace bytes of moe_latent_layer for up to max_tokens tokens (0 if the
 * descriptor is invalid or unsupported); 256-byte aligned, no
 * initialisation needed, nothing in it a caller reads. */
size_t moe_latent_workspace_bytes(const moe_latent_desc *desc, int32_t max_tokens);

/* The expert path a moe_latent_layer call with T tokens takes. */
int32_t moe_latent_path_for(const moe_latent_desc *desc, int32_t T);

/*
 * The latent layer.  x: [T][H] bf16 bits (16-byte aligned); out_bf16 / out_f32
 * [T][H] as out_mode asks (bf16 = round to nearest even of the fp32 result);
 * ids_opt / weights_opt ([T][k], the routing as moe_route orders it) and
 * counts_opt ([E]) receive the routing when non-NULL.
 */
moe_status moe_latent_layer(const moe_latent_desc *desc, const uint16_t *x, int32_t T,
                            uint16_t *out_bf16, float *out_f32, int32_t out_mode,
                            int32_t *ids_opt, float *weights_opt, int32_t *counts_opt,
                            void *ws, size_t ws_bytes, void *stream);

/*
 * moe_latent_layer with phase timing (results equal bit for bit): events[0]
 * before the first launch, [1] after the full-width front (router logits,
 * z, the shared experts' gate/up), [2] after top-k, dispatch and the fp16 z,
 * [3] after the routed gate/up, [4] after the routed down, [5] after the
 * aggregate, its norm, the up projection, the shared experts' down and the
 * output.
 */
moe_status moe_latent_layer_timed(const moe_latent_desc *desc, const uint16_t *x, int32_t T,
                                  uint16_t *out_bf16, float *out_f32, int32_t out_mode,
                                  void *ws, size_t ws_bytes, void *stream, void *const *events);

/*
 * Routing in its other usual forms, from router logits the caller computed:
 * softmax or sigmoid scores, a selection bias, groups of experts of which
 * only the best are considered, top-k, renormalised and scaled weights.
 *
 *   score:   s_e = 1 / (1 + exp(-l_e))                       (MOE_SCORE_SIGMOID)
 *            s_e = exp(l_e) / sum_i exp(l_i)                 (MOE_SCORE_SOFTMAX)
 *   chosen by c_e = s_e + bias_e (the bias steers selection only);
 *   groups:  expert e is in group e / (E / n_groups); a group's value is its
 *            largest c (MOE_GROUP_MAX) or the sum of its two largest
 *            (MOE_GROUP_TOP2; of its only one where it has no second); the
 *            top_groups groups of the largest values stay, ties to the lower
 *            group;
 *   top-k:   the k experts of the largest c in them, descending, ties to the
 *            lower id;
 *   weight_j = s[id_j] / sum_j s[id_j] (if renorm; 0 if that sum is 0)
 *              * routed_scale.
 *
 * Scores, selection and weights are computed in 64 bits, the weights rounded
 * to fp32 once, so two experts tie only where their c are equal as doubles.
 *
 * An expert whose logit or bias is -inf takes no part: not in the softmax's
 * sum, not in its group's value, never chosen.  Where fewer than k experts
 * are left the remaining places hold id -1 and weight 0 (moe_expert_forward
 * drops such terms).  A logit of +inf is the limit (softmax: the experts at
 * +inf share the whole).  A NaN logit makes its own score NaN (softmax: every
 * score of its token); a NaN c ranks with +inf, so it is chosen and its NaN
 * weight shows.
 */
/* (MOE_MXFP4: operands of moe_grouped_linear only) */
typedef enum { MOE_BF16 = 0, MOE_F16 = 1, MOE_F32 = 2, MOE_MXFP4 = 3 } moe_type;
typedef enum { MOE_SCORE_SIGMOID = 0, MOE_SCORE_SOFTMAX = 1 } moe_score;
typedef enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 } moe_group_score;

/* Supported: 1 <= top_k <= E <= 1024, top_k <= 64, n_groups <= 64; E a
 * multiple of n_groups, 1 <= top_groups <= n_groups and top_k <= the experts
 * of top_groups groups (otherwise MOE_EINVAL). */
typedef struct {
    int32_t n_experts, top_k;
    int32_t score;               /* moe_score                                    */
    int32_t n_groups, top_groups;/* 1, 1: no groups                              */
    int32_t group_score;         /* moe_group_score                              */
    int32_t renorm;              /* 1: weights renormalised to sum to 1          */
    float routed_scale;          /* multiplies every weight                      */
    const float *bias;           /* [E] fp32 selection bias, or NULL for none    */
} moe_gate_desc;

/*
 * logits: T rows of E values of logits_type (moe_type), row t at
 * logits + t * ld (ld in elements, >= E; element alignment is enough).
 * ids, weights: [T][k]; counts: [E] or NULL, as moe_route writes them.
 * Needs no workspace.  The same call always gives the same bits.
 */
moe_status moe_gate(const moe_gate_desc *gate, const void *logits, int32_t logits_type,
                    int64_t ld, int32_t T, int32_t *ids, float *weights, int32_t *counts,
                    void *stream);

/*
 * moe_route with the scores, groups, bias, renormalisation and scale of
 * `gate` (desc's own router_bias, renorm and routed_scale are not read):
 * the fp32 logits of x with desc->router_w, computed as moe_route does, then
 * moe_gate on them.  gate and desc have to agree on n_experts and top_k.
 * Workspace as for moe_route.
 */
moe_status moe_route_gated(const moe_layer_desc *desc, const moe_gate_desc *gate,
                           const uint16_t *x, int32_t T, int32_t *ids, float *weights,
                           int32_t *counts, void *ws, size_t ws_bytes, void *stream);

/*
 * Dense product with its epilogue, for the layers around the experts (router
 * logits, projections, dense and shared FFNs):
 *
 *   a[t][n] = sum_k x[t][k] * w[n][k] + bias[n]
 *   u[t][n] = sum_k x[t][k] * w_up[n][k] + bias_up[n]    (gated activations)
 *   out[t][n] = act(a[t][n] (, u[t][n])) + residual[t][n]
 *
 *   MOE_LINEAR_NONE a, RELU max(a, 0), SILU a sigmoid(a),
 *   GELU a Phi(a) = a erfc(-a / sqrt 2) / 2,
 *   GELU_TANH a (1 + tanh(sqrt(2 / pi) (a + 0.044715 a^3))) / 2,
 *   gated: SITU_GLU and SWIGLU, moe_act's SiTU-GLU and SwiGLU of (a, u).
 *
 * x, w, w_up and the 16-bit output have desc->type (MOE_BF16 or MOE_F16);
 * the sums, the epilogue and the fp32 output are fp32, the 16-bit output one
 * round to nearest even of it.  A single token takes the same call.
 */
typedef enum {
    MOE_LINEAR_NONE = 0, MOE_LINEAR_RELU = 1, MOE_LINEAR_SILU = 2, MOE_LINEAR_GELU = 3,
    MOE_LINEAR_GELU_TANH = 4, MOE_LINEAR_SITU_GLU = 5, MOE_LINEAR_SWIGLU = 6
} moe_linear_act;

/* Supported: 1 <= n_in, n_out <= 2^20, n_in <= ldw <= 2^22.  Elements need
 * their own alignment only; rows that are 16-byte aligned (pointers and
 * leading dimensions) with n_in a multiple of 8 take the faster kernels. */
typedef struct {
    int32_t n_in, n_out;
    int32_t type;            /* moe_type of x, w, w_up and the 16-bit output      */
    int32_t act;             /* moe_linear_act                                   */
    float situ_b1, situ_b2;  /* SiTU betas; unused otherwise                      */
    int32_t bias_type;       /* MOE_F32 or `type`                                */
    int32_t residual_type;   /* MOE_F32 or `type`                                */
    int64_t ldw;             /* elements between rows of w and of w_up            */
    const void *w;           /* [n_out][n_in]                                    */
    const void *w_up;        /* [n_out][n_in], for the gated activations only     */
    const void *bias;        /* [n_out], or NULL                                 */
    const void *bias_up;     /* [n_out], or NULL (gated activations only)         */
} moe_linear_desc;

/* Workspace bytes of moe_linear for up to max_tokens tokens (0 if the
 * descriptor is invalid or unsupported); 256-byte aligned, no initialisation
 * needed, nothing in it a caller reads. */
size_t moe_linear_workspace_bytes(const moe_linear_desc *desc, int32_t max_tokens);

/* The kernel that moe_linear takes for T >= 1 tokens whose rows start at x,
 * ldx apart (its arguments), as a moe_linear_path + 256 * the parts that n_in
 * is split into; a negative moe_status for a call it refuses.  Launches
 * nothing and reads nothing behind the pointers.  ROWS16: 16 weight rows a
 * block and 8, 16 or 32 tokens; TILE, ANY: weight rows x tokens, ANY where
 * rows of x or w are not 16-byte aligned (TILE256X128: of moe_mx_linear and
 * moe_grouped_linear only). */
typedef enum {
    MOE_LINEAR_ROWS16X8 = 0, MOE_LINEAR_ROWS16X16 = 1, MOE_LINEAR_ROWS16X32 = 2, MOE_LINEAR_TILE64X32 = 3,
    MOE_LINEAR_TILE64X64 = 4, MOE_LINEAR_TILE128X64 = 5, MOE_LINEAR_TILE128X128 = 6, MOE_LINEAR_ANY64X32 = 7,
    MOE_LINEAR_ANY64X64 = 8, MOE_LINEAR_ANY128X128 = 9, MOE_LINEAR_TILE256X256 = 10, MOE_LINEAR_TILE256X128 = 11
} moe_linear_path;
int32_t moe_linear_path_for(const moe_linear_desc *desc, const void *x, int64_t ldx, int32_t T);

/*
 * x: T rows of n_in values, ldx >= n_in elements apart.  residual: NULL, or T
 * rows of n_out values, ldr elements apart, ldr >= n_out or 0 (the same row
 * for every token).  out_mode: MOE_OUT_BF16 writes out_half (the 16-bit
 * output, in desc->type), MOE_OUT_F32 out_f32, MOE_OUT_BOTH both; rows ldo >=
 * n_out elements apart, the elements between them left as they are.  ldx, ldr
 * and ldo go up to 2^22 (MOE_EUNSUPPORTED above) where there are two rows or
 * more; a single row may lie in rows of any length.
 * An output may be the residual's own buffer (same pointer, row distance and
 * type); otherwise outputs must not overlap inputs.
 */
moe_status moe_linear(const moe_linear_desc *desc, const void *x, int64_t ldx, int32_t T,
                      const void *residual, int64_t ldr, void *out_half, float *out_f32,
                      int64_t ldo, int32_t out_mode, void *ws, size_t ws_bytes, void *stream);

/*
 * MXFP4 rows: codes and scales as moe_layer_desc's (the low nibble first, one
 * E8M0 byte per 32 values of a row), made and read back.
 *
 *   block of 32 values, the last one of a row filled up with zeros:
 *   e = floor(log2(largest magnitude)) - 2      (MOE_MX_FLOOR, the format's own
 *                                                rule: magnitudes past 6 * 2^e
 *                                                become 6 * 2^e), or
 *   e = the least with largest magnitude <= 6 * 2^e                (MOE_MX_FIT),
 *   and at least -127 in both; scale byte e + 127;
 *   code = value / 2^e as E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), round
 *   to nearest, ties to the even code.
 *
 * A block without a value but zeros has scale byte 0.  One with an infinity
 * or a NaN has byte 255 and codes of 0: moe_mx_dequantize reads NaN for its
 * values, a product with them is NaN (and a layer, as moe_layer_desc says,
 * drops the block).  Reading back is exact but for fp32 outputs' overflow to
 * infinity and fp16's rounding, range and subnormals.
 */
typedef enum { MOE_MX_FLOOR = 0, MOE_MX_FIT = 1 } moe_mx_rule;

/*
 * x: T rows of n values of `type` (moe_type), ldx elements apart.  codes: rows
 * of 16 ceil(n / 32) bytes, ldc bytes apart; scales: rows of ceil(n / 32)
 * bytes, lds bytes apart; bytes between rows stay as they are.  Elements need
 * their own alignment only.  1 <= n <= 2^20.  Weights of several experts are
 * rows one after the other.
 */
moe_status moe_mx_quantize(const void *x, int32_t type, int64_t ldx, int32_t T, int32_t n, int32_t rule, uint8_t *codes,
                           int64_t ldc, uint8_t *scales, int64_t lds, void *stream);

/* The values of such rows: out, T rows of n values of `type`, ldo elements apart. */
moe_status moe_mx_dequantize(const uint8_t *codes, int64_t ldc, const uint8_t *scales, int64_t lds, int32_t T, int32_t n, void *out,
                             int32_t type, int64_t ldo, void *stream);

/*
 * moe_linear on MXFP4 rows x, w, w_up: the same formula, activations, biases,
 * residual and outputs.  A product of 128 codes of a row is summed as the
 * matrix cores do, terms below about 2^-24 of its largest one cut off; the
 * rest as moe_linear.  Scale byte 255 is NaN (0 in the layer).
 *
 * n_in is a multiple of 32 (moe_mx_quantize fills up other rows: n_in is then
 * the next one).  Rows of codes start at multiples of 16 bytes, scales
 * anywhere; where n_in is no multiple of 128 or scale rows do not start at
 * multiples of 4 bytes, a launch before the product copies them into the
 * workspace.
 */
typedef struct {
    int32_t n_in, n_out;
    int32_t type;            /* moe_type of the 16-bit output: MOE_BF16, MOE_F16  */
    int32_t act;             /* moe_linear_act                                   */
    float situ_b1, situ_b2;  /* SiTU betas; unused otherwise                      */
    int32_t bias_type;       /* MOE_F32 or `type`                                */
    int32_t residual_type;   /* MOE_F32 or `type`                                */
    int64_t ldw, ldw_s;      /* bytes between rows of codes, of scales            */
    const uint8_t *w, *w_up;     /* [n_out][n_in / 2]; w_up: gated activations    */
    const uint8_t *w_s, *w_up_s; /* [n_out][n_in / 32]                           */
    const void *bias, *bias_up;  /* as moe_linear_desc                           */
} moe_mx_linear_desc;

/* As moe_linear's.  The kernels are moe_linear's too (moe_linear_path; never
 * one of ANY). */
size_t moe_mx_linear_workspace_bytes(const moe_mx_linear_desc *desc, int32_t max_tokens);
int32_t moe_mx_linear_path_for(const moe_mx_linear_desc *desc, int32_t T);

/* x, x_s: T rows of codes and of scales, ldx and ldxs bytes apart (up to 2^23
 * and 2^22); the rest as moe_linear. */
moe_status moe_mx_linear(const moe_mx_linear_desc *desc, const uint8_t *x, int64_t ldx, const uint8_t *x_s, int64_t ldxs, int32_t T,
                         const void *residual, int64_t ldr, void *out_half, float *out_f32, int64_t ldo, int32_t out_mode,
                         void *ws, size_t ws_bytes, void *stream);

/*
 * Experts of other precisions than the layer's, one product at a time: the
 * choices of a routing sorted by expert (moe_group), the products of each
 * expert's rows with its weights (moe_grouped_linear), and the rows of each
 * token added up (moe_combine).
 * The products' rows are what the matrix cores take, 16-bit or MXFP4 ones, so
 * the hidden rows between two products of an FFN are rounded to them; rows that
 * are to be added up can stay in fp32 (MOE_OUT_F32).
 *
 * moe_group: ids [T][k] as moe_gate writes them (an id outside [0, n_experts)
 * is no choice; the same id may come again in a row).  Rows, one per choice,
 * are sorted by expert and inside one by (token, choice):
 *   offsets[n_experts + 1]: expert e's are offsets[e] .. offsets[e + 1] - 1;
 *   tokens[T k]: the token of each row (the places from offsets[n_experts] on
 *   are left as they are);
 *   places[T][k]: the row of each choice, -1 for none.
 * n_experts up to 1024, k up to 64.  Workspace as moe_linear's.  The outputs
 * must not overlap ids or each other.
 */
size_t moe_group_workspace_bytes(int32_t max_tokens, int32_t top_k, int32_t n_experts);
moe_status moe_group(const int32_t *ids, int32_t T, int32_t top_k, int32_t n_experts, int32_t *offsets, int32_t *tokens,
                     int32_t *places, void *ws, size_t ws_bytes, void *stream);

/*
 * out[r] = act(sum_k x[rows[r]][k] w[g][n][k] + bias[g][n] (, the same of w_up))
 * for the rows r of group g, offsets[g] <= r < offsets[g + 1]; activations and
 * sums as moe_linear's (MXFP4: as moe_mx_linear's).
 */
typedef struct {
    int32_t n_groups, n_in, n_out;   /* up to 1024, 2^20, 2^20                    */
    int32_t type;            /* MOE_BF16 or MOE_F16: 16-bit operands and output   */
    int32_t operands;        /* moe_type of x, w, w_up: `type` or MOE_MXFP4       */
    int32_t act;             /* moe_linear_act                                   */
    float situ_b1, situ_b2;  /* SiTU betas; unused otherwise                      */
    int32_t bias_type;       /* MOE_F32 or `type`                                */
    int64_t ldw, group_w;    /* elements (MXFP4: bytes) between rows of w and w_up,
                                and between groups' matrices (>= 0)               */
    int64_t ldw_s, group_w_s;/* MXFP4: bytes between rows of scales, and groups'  */
    const void *w, *w_up;    /* [n_groups][n_out][n_in]                          */
    const uint8_t *w_s, *w_up_s; /* MXFP4: [n_groups][n_out][n_in / 32]          */
    const void *bias, *bias_up;  /* [n_groups][n_out], or NULL                   */
} moe_grouped_desc;

/* The kernel that moe_grouped_linear takes for R >= 1 rows from an x at this
 * address with this row distance (n_in where x has one row): a moe_linear_path
 * + 256. */
int32_t moe_grouped_path_for(const moe_grouped_desc *desc, const void *x, int64_t ldx, int32_t R);

/*
 * x: x_rows rows of n_in values, ldx elements (MXFP4: bytes; x_s, ldxs the
 * scales' rows; both NULL / unused otherwise) apart.  rows: [R] the row of x
 * behind each row, a row of zeros for one outside [0, x_rows); or NULL: row r
 * is x's own (x_rows >= R).  offsets: [n_groups + 1], not decreasing; rows
 * before offsets[0] and from min(offsets[n_groups], R) on are left as they
 * are.  Offsets outside [0, R] count as its ends (where they decrease, which
 * rows are written is not defined; none outside [0, R) is).  rows and offsets
 * are read on the device, so the call needs no synchronisation behind moe_group.
 *
 * 0 <= R <= 2^24; ldx, ldw, ldo up to 2^22 (MXFP4: ldx, ldw up to 2^23, ldxs,
 * ldw_s to 2^22); with `rows`, x's rows lie within 2 GiB; a launch holds fewer
 * than 2^32 threads (n_out (R / 128 + n_groups) below 2^28 always does;
 * MOE_EUNSUPPORTED where none can).  MXFP4: n_in a multiple of 128, rows of
 * codes at multiples of 16 bytes, rows of scales at multiples of 4
 * (MOE_EUNSUPPORTED for n_in and the scales); rows of another width lie in
 * zeroed ones of such a width, since moe_mx_quantize takes row distances, and
 * codes and scale bytes of 0 add nothing.  16-bit elements need their own
 * alignment only; rows at multiples of 16 bytes, n_in of 8, take the faster
 * kernels.  Outputs as moe_linear's; they must not overlap inputs.
 * Needs no workspace.
 */
moe_status moe_grouped_linear(const moe_grouped_desc *desc, const void *x, int64_t ldx, const uint8_t *x_s, int64_t ldxs,
                              int32_t x_rows, const int32_t *rows, const int32_t *offsets, int32_t R, void *out_half,
                              float *out_f32, int64_t ldo, int32_t out_mode, void *stream);

/*
 * out[t][i] = sum_j weights[t][j] y[places[t][j]][i] + residual[t][i], j in its
 * order, in fp32, rounded once.  y: R rows of n values, ldy elements apart; a
 * place outside [0, R) adds nothing.  weights: [T][k] fp32, or NULL for 1.
 * residual: NULL, or T rows ldr apart (0: the same row for every token).
 * y, residual and out (rows ldo apart) each have a moe_type of their own
 * (MOE_BF16, MOE_F16, MOE_F32).  out may be the residual's own buffer (same
 * pointer, row distance and type); otherwise it must not overlap inputs.  k up
 * to 64, n up to 2^20.
 */
moe_status moe_combine(const void *y, int32_t y_type, int64_t ldy, int32_t R, const int32_t *places, const float *weights, int32_t T,
                       int32_t top_k, int32_t n, const void *residual, int32_t residual_type, int64_t ldr, void *out,
                       int32_t out_type, int64_t ldo, void *stream);

/* Static text for a status code. */
const char *moe_status_str(int32_t status);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H */
