/*
 * epdc_layer.h -- C ABI of libepdc_layer.so: the operators of a
 * mixture-of-experts layer on both sides of dispatch and combine (epdc.h).
 *
 *   gate              router logits -> the experts and weights dispatch takes,
 *                     with per-expert counts and the balance and z losses
 *   gate_backward     their gradient with respect to the logits
 *   expert_product    the experts' matrix products over the received rows,
 *                     with bias, activation and residual in the epilogue
 *   expert_backward   their gradients: input rows, weights, biases
 *   combine_backward  combine's gradients: expert rows and routing weights
 *
 * (The gradient of dispatch is epdc_combine with weights NULL: the sum of a
 * token's K gradient rows.)
 *
 * The received layout is that of epdc.h: rows grouped by expert, experts
 * ascending; expert e owns rows [expert_off[e], expert_off[e+1]).
 *
 * Conventions for every entry point:
 *  - Pointers are device addresses on the current device; the caller
 *    allocates and owns all of them.  The library allocates nothing.
 *  - `stream` is a hipStream_t passed as void*; NULL is the null stream.  The
 *    work is enqueued on it and the call returns without waiting.  No call
 *    records a memset node, so every one can be captured into a HIP graph.
 *  - Row-major layouts, no padding between rows.  Logits, payload rows (input,
 *    weight, residual, preact, out), gradients of them and the products' bias
 *    start 16-byte aligned, every other array 4-byte aligned.
 *  - A call with no rows or tokens enqueues what its outputs need (zeroed
 *    losses and counts, zero weight gradients) and nothing else.
 *  - Sums, softmax statistics and losses are kept in fp32 (the matrix products
 *    in the matrix cores' fp32 accumulators); results are rounded once, to
 *    nearest even.  Every result is deterministic: no floating-point atomics.
 *  - Status codes are those of epdc.h; epdc_layer_last_error() gives a
 *    thread-local message.  A status other than SUCCESS leaves no work
 *    enqueued, except EPDC_ERR_GPU_OP after a failed launch.
 */
#ifndef EPDC_LAYER_H
#define EPDC_LAYER_H

#include <stddef.h>
#include <stdint.h>

#include "epdc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of logits and matrix operands. */
typedef enum epdc_layer_dtype {
    EPDC_DT_BF16 = 0,
    EPDC_DT_FP32 = 1,   /* logits and weight gradients only */
    EPDC_DT_E4M3 = 2    /* OCP E4M3 with fp32 scales: product operands only */
} epdc_layer_dtype;

/* The score a gate takes of its logits. */
typedef enum epdc_gate_score {
    EPDC_GATE_SOFTMAX = 0,
    EPDC_GATE_SIGMOID = 1
} epdc_gate_score;

/* Activation of a product's epilogue.  The gated ones take the first half of
 * the weight's rows as gate and the second half as up, and halve the output:
 * out = act(gate) * up. */
typedef enum epdc_activation {
    EPDC_ACT_NONE = 0,
    EPDC_ACT_RELU = 1,
    EPDC_ACT_GELU = 2,     /* with the error function */
    EPDC_ACT_SILU = 3,
    EPDC_ACT_SWIGLU = 4,   /* silu(gate) * up */
    EPDC_ACT_GEGLU = 5     /* gelu(gate) * up */
} epdc_activation;

/*
 * gate.  Per token t, with l = logits[t, :]:
 *   score    s = softmax(l) or sigmoid(l)
 *   choice   the topk experts with the largest s + bias (bias NULL: largest
 *            l), largest first, ties to the lowest index.  With a bias the
 *            order is that of the exact values: keys too close for fp32 are
 *            compared again in 64 bits.
 *   weights  scale * s[choice], divided by the sum of the chosen s when
 *            `renormalize`; the bias never enters them.
 * A logit of -inf makes its expert unavailable.  Where fewer than topk experts
 * are available the remaining entries get index -1 and weight 0.  A token
 * with mask 0, or with no available expert, gets only such entries and takes
 * part in nothing else, whatever its logits hold.  A logit of NaN or +inf in
 * any other token gives it indices -1 and weights NaN, and NaN losses.
 * epdc_dispatch gives a pair of index -1 no slot, raises bit 1 of its
 * device error flag as for any id outside [0, E), and combine adds
 * nothing for it.
 *
 * Balance (counts, losses and scratch all given, or all NULL), over the n
 * tokens that take part and c[e] choices of expert e:
 *   counts [num_experts + 1] = c[0..E-1], n
 *   losses [2] = E * sum_e c[e]/(n*topk) * mean_t p[t, e],  mean_t lse(l)^2
 * with p = s for softmax, s / sum(s) for sigmoid; both 0 for n = 0.
 */
typedef struct epdc_gate_args {
    int32_t num_tokens;     /* >= 0, num_tokens * num_experts < 2^40 */
    int32_t num_experts;    /* [1, 512] */
    int32_t topk;           /* [1, 16], <= num_experts */
    int32_t score;          /* epdc_gate_score */
    int32_t renormalize;    /* 0 or 1 */
    int32_t logits_dtype;   /* EPDC_DT_FP32 or EPDC_DT_BF16 */
    float scale;
    const void *logits;     /* [T, E] */
    const float *bias;      /* [E] or NULL */
    const uint8_t *mask;    /* [T] or NULL: 0 = padding */
} epdc_gate_args;

/* Bytes of scratch a balance needs for up to max_tokens tokens (host only).
 * The caller zero-fills it once; every call leaves it ready for the next.
 * Calls that share a scratch must be ordered. */
epdc_status epdc_gate_scratch_bytes(int32_t max_tokens, int32_t num_experts, size_t *bytes);

epdc_status epdc_gate(const epdc_gate_args *args, void *stream, float *weights, int32_t *indices,
                      int32_t *counts, float *losses, void *scratch);

/*
 * Gradient of the gate.  args as in the forward (the bias does not enter: the
 * choice has no gradient).
 *   indices       [T, K] of the forward
 *   grad_weights  [T, K] fp32 or NULL
 *   counts, grad_losses  [E + 1] of the forward and [2] fp32, or both NULL
 *   grad_logits   [T, E] in the logits' dtype, every entry written: 0 for
 *                 tokens that take part in nothing and for unavailable experts
 * Expert counts are constants of the balance loss's gradient.
 */
epdc_status epdc_gate_backward(const epdc_gate_args *args, void *stream, const int32_t *indices,
                               const float *grad_weights, const int32_t *counts,
                               const float *grad_losses, void *grad_logits);

/*
 * expert_product: for every row s of expert e (row range clamped to [0, rows)),
 *   z = input[s, :] . weight[e]^T + bias[e]
 *   out[s, :] = round(act(z) + residual[s, :])
 * Rows outside [expert_off[0], expert_off[num_experts]) are left as they were.
 * Each call is one launch of fewer than 2^32 threads (512 for a tile of 256
 * columns by 64 or 256 rows, 256 for one of 16 columns by 16 or 32 rows); a
 * call of more tiles is refused.
 *   bf16: in_features and out_features multiples of 8 (gated: out_features a
 *         multiple of 16).
 *   e4m3: in_features a multiple of 128; scales [rows, in/128] fp32 (the
 *         layout dispatch writes), weight_scales [E, ceil(out/128), in/128]
 *         fp32, one per block of 128 x 128; bias, residual and out as in bf16.
 *         The matrix cores add the products of 8 consecutive features after
 *         cutting each off (toward zero) at 2^-13 of the largest exponent
 *         among them; everything above that, the blocks' scales included, is
 *         fp32.
 */
typedef struct epdc_product_args {
    int32_t rows;            /* [0, 2^30]: rows of input, out, residual, preact */
    int32_t num_experts;     /* [1, 512]: experts of weight, bias, expert_off */
    int32_t in_features;     /* [8, 2^20] */
    int32_t out_features;    /* [8, 2^20]: rows of weight (both halves of a gated one) */
    int32_t dtype;           /* EPDC_DT_BF16 or EPDC_DT_E4M3 */
    int32_t activation;      /* epdc_activation */
    int32_t expected_rows;   /* rows these experts are likely to hold, 0 = all `rows`:
                                decides which form runs fastest, nothing else */
    const void *input;       /* [rows, in] */
    const float *scales;     /* e4m3: [rows, in/128], else NULL */
    const void *weight;      /* [E, out, in] */
    const float *weight_scales; /* e4m3: [E, ceil(out/128), in/128], else NULL */
    const float *bias;       /* [E, out] fp32 or NULL */
    const int32_t *expert_off;  /* [E + 1], ascending */
} epdc_product_args;

/* residual [rows, cols] bf16 or NULL; out [rows, cols] bf16, cols = out_features
 * (gated: half of it); preact [rows, out_features] bf16 or NULL: z, rounded, for
 * expert_backward.  out and preact may overlap neither each other nor an input,
 * except that out may be residual itself. */
epdc_status epdc_expert_product(const epdc_product_args *args, void *stream, const void *residual,
                                void *out, void *preact);

/*
 * expert_backward (bf16).  With dz = grad_out * act'(preact) (grad_out itself
 * without an activation), rounded to bf16 for the two products:
 *   grad_input[s, :]  = dz[s, :] . weight[e]              or NULL
 *   grad_weight[e]    = sum_s dz[s, :]^T input[s, :]      or NULL
 *   grad_bias[e]      = sum_s dz[s, :] (not rounded)      or NULL (fp32)
 * grad_weight and grad_bias are written for every expert, zeros where it has
 * no rows; grad_input only for the experts' rows.  residual's gradient is
 * grad_out.
 *   preact       [rows, out_features] bf16, NULL for EPDC_ACT_NONE
 *   dz           [rows, out_features] bf16 workspace; NULL for EPDC_ACT_NONE, or
 *                when only grad_bias is asked for
 *   grad_weight  [E, out, in] in grad_weight_dtype (EPDC_DT_BF16 or EPDC_DT_FP32)
 * Outputs and dz may overlap neither each other nor anything the call reads;
 * without grad_bias dz may be preact itself or (not gated) grad_out itself.
 */
epdc_status epdc_expert_backward(const epdc_product_args *args, void *stream,
                                 const void *grad_out, const void *preact, void *dz,
                                 void *grad_input, void *grad_weight, int32_t grad_weight_dtype,
                                 float *grad_bias);

/*
 * combine_backward: for every pair (t, k) with a slot s = slot_of[t*K + k] in
 * [0, num_tokens*topk),
 *   grad_input[s, :]   = round(w * grad_output[t, :]),  w = weights[s, k] (1 if NULL)
 *   grad_weights[t, k] = sum_h grad_output[t, h] * input[s, h]
 * A pair without a slot gets grad_weights 0; rows without a pair are left as
 * they were.  slot_of is epdc_get_routing's.  grad_weights may be NULL (input
 * is then not read and may be NULL); grad_input may be NULL.  The outputs may
 * overlap neither each other nor an input, except that grad_input may be input.
 */
epdc_status epdc_combine_backward(void *stream, int32_t num_tokens, int32_t topk, int32_t hidden,
                                  const int32_t *slot_of, const void *grad_output,
                                  const void *input, const float *weights, void *grad_input,
                                  float *grad_weights);

/* Thread-local message for the last non-SUCCESS status ("" if none). */
const char *epdc_layer_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* EPDC_LAYER_H */
