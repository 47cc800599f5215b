/*
 * moe_layer.h -- C ABI of the operators around MoE routing: the router's balance loss and the
 * gradient of its logits, 8-bit rows with a scale for each token, and the experts' product in
 * 8-bit integers. Part of the same library as moe_route.h, whose rows they read and write:
 *
 *   serving   moe_quant_rows(x) -> moe_expert_matmul_i8 (gate and up, SwiGLU) over the rows of
 *             moe_dispatch_layout -> moe_quant_rows -> moe_expert_matmul_i8 (down) -> moe_combine;
 *   training  moe_route_topk -> moe_balance_loss, and moe_route_grad for the logits.
 *
 * The conventions of moe_route.h hold: device pointers, caller-owned buffers, no allocation and no
 * state, work enqueued on `stream`, arguments validated before any launch, dense row-major
 * matrices, and no access outside the buffers whatever the values of ids, rows and offsets.
 */
#ifndef MOE_LAYER_H
#define MOE_LAYER_H

#include "moe_route.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Balance loss. The batch is S = n_seqs sequences of L = T / S consecutive tokens (S = 1: the loss
 * over the whole batch). token_mask [T] uint8 may be NULL; a token with mask 0 is padding and
 * counts nowhere. For sequence s with n_s unmasked tokens,
 *   p_t     = softmax of row t of logits over all E experts (a logit of -infinity has p = 0; a row
 *             of nothing else has p = 0 everywhere; a row with a NaN or +infinity gives NaN),
 *   c_se    = slots (t, j) of unmasked tokens with topk_idx = e (ids outside [0, E) are skipped),
 *   P_se    = sum of p_te over the unmasked tokens,
 *   loss[0] = alpha / S * sum_s E / (k * n_s^2) * sum_e c_se * P_se   (n_s = 0 adds 0),
 * so loss = alpha for perfectly even routing. With f_se = c_se E / (k n_s) this is
 * alpha / S * sum_s sum_e f_se * mean_t p_te.
 *   logits        [T, E] fp32, topk_idx [T, k] int32 (as written by moe_route_topk).
 *   loss          [1] fp32 out, expert_counts [S, E] int32 out, prob_sums [S, E] fp32 out,
 *   seq_tokens    [S] int32 out: n_s. Counts and tokens are what moe_route_grad takes.
 *   workspace     moe_balance_workspace_bytes(T, E, S) bytes, 16-byte aligned, any contents; calls
 *                 that may run at the same time must not share one.
 * p and the sums of a workgroup are fp32, sums over workgroups and the loss fp64; every order is
 * fixed, so equal inputs give equal bits. Requires T % S == 0, T * k < 2^31, 1 <= S, E, k (else
 * MOE_ERR_INVALID), S <= MOE_MAX_SEQS, E <= MOE_MAX_EXPERTS and k <= MOE_MAX_TOPK (else
 * MOE_ERR_UNSUPPORTED). T = 0 writes zeros.
 */
#define MOE_MAX_SEQS 65536

size_t moe_balance_workspace_bytes(int32_t T, int32_t E, int32_t n_seqs);

moe_status_t moe_balance_loss(const float* logits, const int32_t* topk_idx,
                              const uint8_t* token_mask, int32_t T, int32_t E, int32_t k,
                              int32_t n_seqs, float alpha, float* loss, int32_t* expert_counts,
                              float* prob_sums, int32_t* seq_tokens, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

/*
 * Gradient of the router's logits: of the balance loss, of the routing weights, or of both.
 *   dlogits[t, e] = g * alpha / S * E / (k * n_s^2) * p_te * (c_se - sum_i c_si p_ti)
 *                   (tokens that are not masked; needs expert_counts and seq_tokens, else absent)
 *                 + sum over slots j with topk_idx[t, j] = e of w_j * (dw_j - sum_i w_i dw_i)
 *                   (all tokens; needs topk_w and dtopk_w, else absent)
 * with g = dloss[0] (fp32 on the device; NULL: 1). The counts are constants of the loss. Counts
 * and tokens may have been summed over devices first: the loss is then that of the joint batch.
 *   topk_w, dtopk_w [T, k] fp32: the weights of moe_route_topk and the gradient that reached them.
 *   topk_idx is read only for the weights; slots outside [0, E) are skipped, equal ids add up.
 *   logits and token_mask are read only for the loss.
 *   dlogits [T, E] fp32 out, every element written.
 * Sizes as for moe_balance_loss; expert_counts and seq_tokens are given together, topk_w and
 * dtopk_w too, and one pair at least (else MOE_ERR_INVALID). T = 0 enqueues nothing.
 */
moe_status_t moe_route_grad(const float* logits, const int32_t* topk_idx, const float* topk_w,
                            const float* dtopk_w, const uint8_t* token_mask,
                            const int32_t* expert_counts, const int32_t* seq_tokens,
                            const float* dloss, int32_t T, int32_t E, int32_t k, int32_t n_seqs,
                            float alpha, float* dlogits, hipStream_t stream);

/*
 * 8-bit rows: for every row, a = max |x|, q = 127 * x / a rounded to the nearest integer (of the
 * exact quotient, ties to even; so |q| <= 127) and scale = a / 127 rounded once to fp32. A row of
 * zeros has q = 0 and scale = 1. A row that holds a NaN or an infinity has q = 0 and scale = NaN,
 * so that everything computed from it is NaN. Below a = 127 * 2^-126 the scale is subnormal and
 * carries its absolute rounding.
 *   x [R, H] x_dtype MOE_F32 or MOE_BF16, 16-byte aligned; q [R, H] int8, 16-byte aligned;
 *   scale [R] fp32. n_rows (device int32 [1], may be NULL): only rows [0, n_rows[0]) are read and
 *   written, the ones behind are left as they were (moe_ep_recv's expert_offsets + L, say).
 * Requires H % 16 == 0 (else MOE_ERR_UNSUPPORTED). R = 0 enqueues nothing.
 */
moe_status_t moe_quant_rows(const void* x, moe_dtype_t x_dtype, int32_t R, int32_t H,
                            const int32_t* n_rows, int8_t* q, float* scale, hipStream_t stream);

#define MOE_MATMUL_MAX_K 131056

typedef enum {
    MOE_ACT_NONE = 0,
    MOE_ACT_SWIGLU = 1   /* silu(gate) * up, with silu(v) = v / (1 + exp(-v)) */
} moe_act_t;

/*
 * The experts' product in 8-bit integers, with a scale for each row and for each output channel:
 *   acc[r, n] = sum_i a[s(r), i] * w[e, n, i]                  (int32, exact)
 *   y[r, n]   = acc[r, n] * a_scale[s(r)] * w_scale[e, n]      (fp32, in this order)
 * for the rows expert_offsets[e] <= r < expert_offsets[e + 1] of expert e, where s(r) =
 * row_token[r], or r if row_token is NULL.
 *   MOE_ACT_NONE    w [E, N, K], out[r, n] = y[r, n].
 *   MOE_ACT_SWIGLU  w [E, 2N, K], gate channels first: out[r, n] = silu(y[r, n]) * y[r, N + n],
 *                   in fp32.
 *   a [a_rows, K] int8, a_scale [a_rows]; w int8, w_scale fp32 per channel of w; both matrices
 *   16-byte aligned. out [R, N] out_dtype MOE_F32 or MOE_BF16 (rounded once, to nearest even).
 *   expert_offsets [E + 1] and row_token [R] are those of moe_dispatch_layout (R = T * k), or of
 *   moe_ep_recv for its L experts (R = S * cap, row_token NULL). NULL expert_offsets: E must be 1
 *   and all R rows are its rows (a plain product). Rows at or behind expert_offsets[E] are left as
 *   they were; so is a row whose row_token lies outside [0, a_rows). Offsets outside [0, R] or
 *   falling break the preconditions and leave the rows of out unspecified.
 * Requires K % 16 == 0 and K <= MOE_MATMUL_MAX_K (the largest for which -128 * -128 * K fits an int32),
 * E <= MOE_MAX_EXPERTS, and one expert's weights and, with row_token, all of `a` below 4 GiB (else
 * MOE_ERR_UNSUPPORTED); R <= a_rows without row_token (else MOE_ERR_INVALID). R = 0 enqueues
 * nothing.
 */
moe_status_t moe_expert_matmul_i8(const int8_t* a, const float* a_scale, int32_t a_rows,
                                  const int32_t* row_token, const int8_t* w, const float* w_scale,
                                  const int32_t* expert_offsets, int32_t R, int32_t E, int32_t N,
                                  int32_t K, moe_act_t act, void* out, moe_dtype_t out_dtype,
                                  hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LAYER_H */
