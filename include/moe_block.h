/*
 * moe_block.h -- C ABI of the rest of a MoE block around routing, in fp32 and bf16: scored routing
 * (softmax or sigmoid, a balance bias, groups of experts) with its gradient and the bias's update,
 * the experts' product with its epilogue and gradients, and the gradient of the weighted combine.
 * Part of the same library as moe_route.h, whose rows they read and write:
 *
 *   forward   moe_expert_matmul (the router's gate: one expert, fp32 out) -> moe_route_scored ->
 *             moe_dispatch_layout -> moe_expert_matmul (gate and up, rows gathered, `pre` kept) ->
 *             moe_expert_matmul (down) -> moe_combine;
 *   backward  moe_combine_grad -> moe_expert_matmul_grad (down, through the activation) ->
 *             moe_expert_matmul_grad (gate and up) -> moe_combine with weights of one for the
 *             tokens; moe_route_scored_grad for the logits, moe_bias_update for the bias.
 *
 * The conventions of moe_route.h hold: device pointers, caller-owned buffers, no allocation and no
 * state, work enqueued on `stream`, arguments validated before any launch, dense row-major
 * matrices, and no access outside the buffers whatever the values of ids, rows and offsets.
 * Outputs must not overlap inputs or each other unless it is said that they may.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_route.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_SCORE_SOFTMAX = 0,   /* s_e = exp(l_e) / sum_i exp(l_i) over all experts */
    MOE_SCORE_SIGMOID = 1    /* s_e = 1 / (1 + exp(-l_e)) */
} moe_score_t;

#define MOE_MAX_GROUPS 64

/*
 * Scored routing. With s the scores of a token and c_e = s_e + bias[e] (bias NULL: c = s):
 *   - the experts form n_groups groups of E / n_groups consecutive ones. A group's score is the sum
 *     of its group_top largest c; the topk_groups groups with the largest scores are kept, equal
 *     ones to the lower number;
 *   - of the experts in kept groups the k with the largest c are chosen, largest first, equal ones
 *     to the lower id;
 *   - topk_w[t, j] = scale * s_j / sum_i s_i over the chosen (renormalize != 0; 0 if the sum is 0),
 *     or scale * s_j. The bias takes part in the choice only.
 * Scores, c, sums and weights are those of 64-bit arithmetic: a choice or a group may go the other
 * way only where two values differ by less than 2^-48 of the larger of |s| and |bias|, and never
 * between experts of equal logits and biases. Weights are rounded once to fp32.
 *   logits [T, E] fp32, bias [E] fp32 or NULL; topk_idx [T, k] int32 out, topk_w [T, k] fp32 out.
 * An expert with a logit of -infinity has s = 0 and is behind every other in the choice, whatever
 * its bias (its c is -infinity, in its group's score too). Ids are always distinct, inside [0, E)
 * and of kept groups. A NaN, a logit of +infinity with MOE_SCORE_SOFTMAX or an infinite bias leaves
 * the row's ids (but for that) and weights unspecified.
 * Requires 1 <= k <= topk_groups * (E / n_groups), E % n_groups == 0, 1 <= topk_groups <= n_groups
 * and 1 <= group_top <= E / n_groups (else MOE_ERR_INVALID), E <= MOE_MAX_EXPERTS, k <= MOE_MAX_TOPK
 * and n_groups <= MOE_MAX_GROUPS (else MOE_ERR_UNSUPPORTED); `scale` finite. With n_groups == 1
 * group_top is not read. T = 0 enqueues nothing.
 */
moe_status_t moe_route_scored(const float* logits, const float* bias, int32_t T, int32_t E,
                              int32_t k, moe_score_t score, int32_t n_groups, int32_t topk_groups,
                              int32_t group_top, int32_t renormalize, float scale,
                              int32_t* topk_idx, float* topk_w, hipStream_t stream);

/*
 * Gradient of the logits through the weights of moe_route_scored, the ids and the bias being
 * constants. For a token with chosen ids e_j, dw_j = dtopk_w[t, j], and S = sum_j s_j:
 *   softmax, renormalized   v_j = s_j / S:  dl_j = scale * v_j * (dw_j - sum_i v_i dw_i)
 *   softmax                 dl_e = scale * s_e * (sum of dw_j with e_j = e - sum_i s_i dw_i), every e
 *   sigmoid, renormalized   dl_j = scale / S * (dw_j - sum_i s_i dw_i / S) * s_j * (1 - s_j)
 *   sigmoid                 dl_j = scale * dw_j * s_j * (1 - s_j)
 *   dlogits[t, e] = sum of dl_j with e_j = e (or dl_e) + add[t, e]
 *   add [T, E] fp32: the gradient that the logits have from elsewhere (moe_route_grad's, say), or
 *   NULL; it may be dlogits itself. dlogits [T, E] fp32 out, every element written.
 * Slots with ids outside [0, E) are left out; equal ids add up. A chosen logit of -infinity has
 * s = 0 and dl = 0. Sizes as for moe_route_scored (k may exceed E). T = 0 enqueues nothing.
 */
moe_status_t moe_route_scored_grad(const float* logits, const int32_t* topk_idx,
                                   const float* dtopk_w, const float* add, int32_t T, int32_t E,
                                   int32_t k, moe_score_t score, int32_t renormalize, float scale,
                                   float* dlogits, hipStream_t stream);

/*
 * Update of the balance biases of L layers:
 *   out[l, e] = bias[l, e] + rate * sign(sum_i expert_counts[l, i] - E * expert_counts[l, e])
 * so an expert above its layer's mean count loses `rate` and one below gains it (one fp32 addition;
 * the comparison is exact). bias, out [L, E] fp32, expert_counts [L, E] int32; out may be bias.
 * Requires L >= 0, E >= 1 (else MOE_ERR_INVALID), E <= MOE_MAX_EXPERTS (else MOE_ERR_UNSUPPORTED).
 */
moe_status_t moe_bias_update(const float* bias, const int32_t* expert_counts, int32_t L, int32_t E,
                             float rate, float* out, hipStream_t stream);

/*
 * Gradient of moe_combine: with row = token_row[t * k + j],
 *   dy[row, h]     = topk_w[t, j] * dout[t, h]           (rounded once to y's type)
 *   dtopk_w[t, j]  = sum_h dout[t, h] * y[row, h]        (fp32, a fixed order)
 *   dout [T, H] dout_dtype, y and dy [T * k, H] y_dtype: MOE_F32 or MOE_BF16 each, 16-byte aligned.
 *   dy or dtopk_w may be NULL (not both): what it would hold is not computed, y and topk_w are not
 *   read for it and may be NULL then. Rows outside [0, T * k) are skipped: dtopk_w is 0 there.
 *   token_row is that of moe_dispatch_layout. Where several slots name one row, an element of dy is that
 *   of any one of them, not their sum.
 * Requires H % 8 == 0 (else MOE_ERR_UNSUPPORTED). Rows that no slot names are left as they were.
 */
moe_status_t moe_combine_grad(const void* dout, moe_dtype_t dout_dtype, const void* y,
                              moe_dtype_t y_dtype, const int32_t* token_row, const float* topk_w,
                              int32_t T, int32_t H, int32_t k, void* dy, float* dtopk_w,
                              hipStream_t stream);

/* Largest K, and largest number of channels of an expert, of the products in bf16. */
#define MOE_MAT_MAX_SIZE 4194304

typedef enum {
    MOE_MAT_NONE = 0,
    MOE_MAT_SWIGLU = 1,   /* silu(gate) * up: the product has 2N channels, gate channels first */
    MOE_MAT_RELU = 2,
    MOE_MAT_SILU = 3,     /* v / (1 + exp(-v)) */
    MOE_MAT_GELU = 4      /* v * (1 + tanh(u)) / 2, u = sqrt(2 / pi) * (v + 0.044715 v^3) */
} moe_mat_act_t;

/*
 * The experts' product in bf16: for the rows expert_offsets[e] <= r < expert_offsets[e + 1] of
 * expert e, where s(r) = row_token[r], or r if row_token is NULL,
 *   y[r, n]   = sum_i a[s(r), i] * w[e, n, i] + bias[e, n]          (fp32)
 *   pre[r, n] = y[r, n]                                             (rounded once to bf16)
 *   out[r, n] = act(y)[r, n] + residual[r, n]                       (fp32, rounded once)
 *   a [a_rows, K] bf16, w [E, N, K] bf16 (MOE_MAT_SWIGLU: [E, 2N, K]), both 16-byte aligned; bias
 *   [E, N or 2N] fp32 or NULL; residual [R, N] of out's type or NULL, it may be out itself;
 *   pre [R, N or 2N] bf16 out or NULL: what moe_expert_matmul_grad needs of the activation;
 *   out [R, N] out_dtype MOE_F32 or MOE_BF16.
 *   expert_offsets [E + 1] and row_token [R] are those of moe_dispatch_layout, or of moe_ep_recv.
 * NULL expert_offsets: E must be 1 and all R rows are its rows (a plain product: the router's gate,
 * a shared expert). Rows at or behind expert_offsets[E] are left as they were in out and pre; so is
 * a row whose row_token lies outside [0, a_rows). Offsets outside [0, R] or falling break the
 * preconditions and leave the rows of the outputs unspecified.
 * Requires K % 8 == 0, K and the channels of w <= MOE_MAT_MAX_SIZE, E <= MOE_MAX_EXPERTS, and one
 * expert's weights and, with row_token, all of `a` below 4 GiB (else MOE_ERR_UNSUPPORTED); R <= a_rows
 * without row_token (else MOE_ERR_INVALID).
 * R = 0 enqueues nothing.
 *   workspace: moe_expert_matmul_workspace_bytes(R, E, channels of w, K) bytes, 16-byte aligned, any
 *   contents, NULL where that is 0 (it is also 0 for sizes that the product refuses); calls that may
 *   run at the same time must not share one. Few tiles with long sums (the gate of a few thousand
 *   tokens) are made in parts, joined in a fixed order.
 */
size_t moe_expert_matmul_workspace_bytes(int32_t R, int32_t E, int32_t channels, int32_t K);

moe_status_t moe_expert_matmul(const void* a, int32_t a_rows, const int32_t* row_token,
                               const void* w, const float* bias, const int32_t* expert_offsets,
                               int32_t R, int32_t E, int32_t N, int32_t K, moe_mat_act_t act,
                               const void* residual, void* pre, void* out, moe_dtype_t out_dtype,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of y[r, n] = sum_i a[s(r), i] * w[e, n, i] + bias[e, n] from dy [R, N] bf16:
 *   da[r, i]    = sum_n dy[r, n] * w[e, n, i]              for every row of an expert
 *   dw[e, n, i] = sum_r dy[r, n] * a[s(r), i]              over the rows of expert e
 *   dbias[e, n] = sum_r dy[r, n]
 * each sum in fp32 and a fixed order, rounded once. da is per row: with row_token, moe_combine with
 * weights of one adds up the rows of a token. Each of da, dw and dbias may be NULL (not all).
 *   act other than MOE_MAT_NONE: a was made as act(pre) and da is the gradient of pre instead,
 *   act'(pre)[r, i] * da[r, i] before its rounding, with pre [R, K] bf16; MOE_MAT_SWIGLU: pre and da
 *   are [R, 2K], gate channels first. relu'(0) = 0. pre is read for da only.
 *   da da_dtype, dw dw_dtype: MOE_F32 or MOE_BF16 each; dbias fp32. a, w, dy, da and dw 16-byte
 *   aligned. w is read for da only, a and row_token's rows for dw only.
 * Rows behind the last expert's, and rows whose row_token lies outside [0, a_rows), are left as
 * they were in da and add nothing to dw and dbias. An expert without rows gets zeros.
 *   workspace: moe_matmul_grad_workspace_bytes(R, E, N, K) bytes, 16-byte aligned, any contents;
 *   calls that may run at the same time must not share one.
 * Requires N % 8 == 0 and K % 8 == 0, and the other limits of moe_expert_matmul. R = 0 writes
 * zeros to dw and dbias.
 */
size_t moe_matmul_grad_workspace_bytes(int32_t R, int32_t E, int32_t N, int32_t K);

moe_status_t moe_expert_matmul_grad(const void* dy, const void* a, int32_t a_rows,
                                    const int32_t* row_token, const void* w,
                                    const int32_t* expert_offsets, int32_t R, int32_t E, int32_t N,
                                    int32_t K, moe_mat_act_t act, const void* pre, void* da,
                                    moe_dtype_t da_dtype, void* dw, moe_dtype_t dw_dtype,
                                    float* dbias, void* workspace, size_t workspace_bytes,
                                    hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
