/*
 * ep_experts.h -- C ABI of libep.so, second part: the steps of an expert layer on either side of
 * the dispatch/combine core of ep.h, on AMD MI355X (gfx950).
 *
 *   ep_route                    router logits -> topk_idx, topk_weights (what ep_get_layout and the
 *                               dispatches take)
 *   ep_route_backward           gradient of topk_weights -> gradient of the logits
 *   ep_expert_gemm_fp8          the experts' product on the grouped rows: E4M3 rows and weights with
 *                               a scale for each block of 128, bf16 out
 *   ep_expert_gemm_swiglu_fp8   gate and up products, silu(gate) * up, and the E4M3 quantiser in one
 *                               launch: what the second product reads
 *   ep_combine_grouped          expert outputs in the grouped layout -> weighted sum in token order
 *   ep_combine_grouped_backward gradient of that sum: of the expert outputs and of topk_weights
 *
 * A layer is  ep_route, ep_layout_notify, ep_quantize_fp8, ep_dispatch_grouped (elem_bytes 1),
 * ep_expert_gemm_swiglu_fp8, ep_expert_gemm_fp8, ep_combine_grouped.
 *
 * The conventions of ep.h hold for every call: device pointers, caller-owned buffers, nothing
 * allocated, no state between calls, kernels enqueued on `stream` only (so every call can be
 * captured in a HIP graph), argument errors reported before any launch, data-dependent problems
 * flagged in *dev_status (nullable) and never trapped.  The calls need no workspace, so calls on
 * different streams share nothing but their inputs.
 */
#ifndef EP_EXPERTS_H
#define EP_EXPERTS_H

#include "ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A further bit of *dev_status. */
enum {
    EP_DEV_BAD_LOGIT = 32 /* a logit that is NaN or +inf, or such a bias: that expert is not routed to */
};

typedef enum { EP_LOGITS_F32 = 0, EP_LOGITS_BF16 = 1 } ep_logits_type_t;
typedef enum { EP_SCORE_SOFTMAX = 0, EP_SCORE_SIGMOID = 1 } ep_score_t;

/* How a router chooses (host struct, read during the call only). */
typedef struct {
    int32_t score;        /* an ep_score_t                                                      */
    int32_t num_groups;   /* G: experts in G groups of E / G consecutive ones; 1 <= G <= 64, G | E */
    int32_t groups_kept;  /* 1..G groups whose experts may be chosen                            */
    int32_t group_best;   /* 1 or 2: a group is rated by the sum of that many best of its experts */
    int32_t renormalize;  /* non-zero: a token's weights are divided by their sum               */
    float weight_scale;   /* finite factor of every weight                                      */
} ep_router_t;

/*
 * Routing to experts.  For token t with logits l_e, e in [0, E):
 *   score   s_e = 1 / (1 + exp(-l_e))                       EP_SCORE_SIGMOID
 *           s_e = exp(l_e) / sum over the token's finite logits of exp(l)   EP_SCORE_SOFTMAX
 *   choice  c_e = s_e + bias_e; with no bias experts are ordered by l_e itself, so that scores
 *           too near 0 or 1 to be told apart make no ties
 *   groups  with G > 1: a group's rating is the sum of its min(group_best, eligible) largest c_e
 *           (its largest l_e when group_best is 1 and there is no bias); the groups_kept groups
 *           of the highest rating stay, ties to the lower group
 *   top k   the num_topk experts of the largest c_e in the groups kept, in descending order,
 *           ties to the lower expert
 *   weight  w_j = weight_scale * s_{e_j}, divided by the sum S of the token's chosen s when
 *           renormalize is set.  A softmax's s_{e_j} / S are formed from the chosen logits alone,
 *           however far they are below the row's largest; a sigmoid's are 0 when every chosen s
 *           is 0 in binary64 (logits below about -709)
 * Choices and ratings compare as in binary64, so near ties are decided as the definition does.
 * Weights are formed in binary64 and rounded to f32 once, but for a softmax that is not
 * renormalised: its denominator is a sum of f32 exponentials, which leaves them within 58 * 2^-24 of
 * their value.  An expert is eligible unless its logit is -inf (a masked
 * expert) or its bias is -inf, or either is NaN or +inf (flagged, EP_DEV_BAD_LOGIT); such an
 * expert is never chosen, and one whose logit is not finite takes no part in the softmax.  Slots
 * that no eligible expert fills, and all slots of a token that token_mask switches off, get
 * topk_idx -1 and weight 0: ep.h's masked slots.
 * In:  logits [t] rows of E values of logits_type, row t at logits + t * logits_stride elements
 *      (logits_stride >= E); bias [E] f32 (nullable); token_mask [t] uint8 (nullable; 0 = the
 *      token is not routed and its logits are not read).
 * Out: topk_idx [t][k] int64, topk_weights [t][k] f32.
 * Limits: num_experts <= 2048, num_tokens <= 2^25 (EP_ERR_UNSUPPORTED).  Logits, bias and
 * topk_weights 4-byte aligned (bf16 logits 2-byte), topk_idx 8-byte aligned.  One launch.
 * dev_status (nullable): EP_DEV_BAD_LOGIT.
 */
ep_status_t ep_route(const ep_shape_t *s, const ep_router_t *r, const void *logits, int32_t logits_type,
                     int64_t logits_stride, const float *bias, const uint8_t *token_mask, int64_t *topk_idx,
                     float *topk_weights, int32_t *dev_status, hipStream_t stream);

/*
 * Gradient of ep_route's weights with respect to the logits; the choice itself has none.  With
 * the token's slots j that hold an expert e_j, S = sum of s_{e_j} and g_j = grad_weights[t][j]:
 *   ds_j = weight_scale * (g_j - sum_i g_i s_{e_i} / S) / S   when renormalize is set
 *   ds_j = weight_scale * g_j                                 otherwise
 *   grad_logits[t][e] = s_e (1 - s_e) * (sum of ds_j over the slots naming e)          sigmoid
 *   grad_logits[t][e] = s_e * (sum of ds_j over the slots naming e - sum_j ds_j s_{e_j})  softmax
 * Each slot's part is formed in binary64 (ds_j is as large as S is small, and is not rounded by
 * itself), with s_{e_j} / S as for the weights: 0 where those are.
 * Slots of -1 have no part (a token whose slots are all -1 gets a row of zeros, and its logits are
 * not read); an expert named by several slots gets the sum.  A logit that is not finite gets 0.
 * In:  logits as ep_route took them; topk_idx [t][k] as it wrote them; grad_weights [t][k] f32.
 * Out: grad_logits, rows of E values of logits_type at a stride of grad_stride elements, written
 *      whole (elements between rows are not touched).  May not overlap logits.
 * Limits as for ep_route (groups and bias play no part).  One launch.
 * dev_status (nullable): EP_DEV_BAD_TOPK_IDX (an id outside [-1, E): that slot is skipped),
 * EP_DEV_BAD_LOGIT.
 */
ep_status_t ep_route_backward(const ep_shape_t *s, const ep_router_t *r, const void *logits, int32_t logits_type,
                              int64_t logits_stride, const int64_t *topk_idx, const float *grad_weights,
                              void *grad_logits, int64_t grad_stride, int32_t *dev_status, hipStream_t stream);

/*
 * The experts' product in E4M3 with a scale for each block of 128, over the grouped rows that
 * ep_dispatch_grouped (elem_bytes 1) or ep_group_by_expert delivers.  Expert e's segment is the
 * expert_rows[e] rows after the segments of the experts before it; for a row m of it and 0 <= c < n:
 *   out[m][c] = bf16(sum over blocks b of (x_scales[m][b] * w_scales[e][c / 128][b])
 *                                          * sum over i in block b of x[m][i] * w[e][c][i])
 * with block b the channels 128 b .. 128 b + 127, both sums in f32, and one rounding to bf16
 * (nearest, ties to even) at the end.
 * In:  x [num_rows][k] E4M3 codes, x_scales [num_rows][k / 128] f32 (ep_quantize_fp8's codes and
 *      scales with num_scales = k / 128); w [num_experts][n][k] E4M3 codes, w_scales
 *      [num_experts][ceil(n / 128)][k / 128] f32; expert_rows [num_experts] int32 (device), as
 *      ep_notify's num_recv_tokens_per_expert (a negative size counts as 0).  expert_rows may be
 *      NULL when num_experts is 1: all num_rows rows are that expert's (a dense product).
 * Out: out [num_rows][n] bf16.  Rows behind the last segment are left as they were, and their x
 *      is not read.
 * The gradient with respect to x's values is the same product of the quantised gradient with the
 * transposed weights: w [num_experts][k][n] and w_scales [num_experts][k / 128][n / 128].
 * Limits: k a positive multiple of 128, n a positive multiple of 8 (EP_ERR_INVALID_ARG); n * k
 * < 2^31, k <= 2^20, num_experts <= 16384, and a launch of no more than 2^31 - 1 threads, 512 for each part
 * of a segment of up to 16 rows and each 64 columns at most (EP_ERR_UNSUPPORTED).
 * x, w and out 16-byte, scales and expert_rows 4-byte aligned.  One launch (with no rows only where
 * there are sizes to look at and a status to set).
 * dev_status (nullable): EP_DEV_RECV_OVERFLOW (the segments pass num_rows, which may be 0: the rows
 * past it are not computed).
 */
ep_status_t ep_expert_gemm_fp8(int32_t num_experts, int32_t n, int32_t k, const void *x, const float *x_scales,
                               const void *w, const float *w_scales, const int32_t *expert_rows, int32_t num_rows,
                               void *out, int32_t *dev_status, hipStream_t stream);

/*
 * Gate and up products, their activation and the quantiser for the second product in one launch.
 * w [num_experts][2 n][k]: rows 0 .. n-1 of an expert are its gate, rows n .. 2n-1 its up matrix;
 * w_scales [num_experts][2 n / 128][k / 128].  With gate and up the products of ep_expert_gemm_fp8
 * before their rounding (f32), for 0 <= c < n:
 *   a[m][c] = gate / (1 + exp(-gate)) * up                                 (f32)
 *   top     = max(largest |a[m][c]| of the block of 128 columns, 2^-64)
 *   out_scales[m][q] = top / 448;  out[m][c] = e4m3(clamp(a[m][c] * (448 / top), -448, 448))
 * as ep_quantize_fp8 has it (nearest, ties to even), so out and out_scales are the x and x_scales
 * of ep_expert_gemm_fp8 with k = n.  (Codes and scale of a block that holds an infinity or NaN are
 * not defined.)
 * Out: out [num_rows][n] uint8 E4M3 codes, out_scales [num_rows][n / 128] f32; rows behind the
 *      last segment are left as they were.
 * Limits: n and k positive multiples of 128 (EP_ERR_INVALID_ARG); 2 n * k < 2^31; the rest, the
 * other arguments, alignment and dev_status as for ep_expert_gemm_fp8.
 */
ep_status_t ep_expert_gemm_swiglu_fp8(int32_t num_experts, int32_t n, int32_t k, const void *x,
                                      const float *x_scales, const void *w, const float *w_scales,
                                      const int32_t *expert_rows, int32_t num_rows, void *out, float *out_scales,
                                      int32_t *dev_status, hipStream_t stream);

/*
 * Combine of expert outputs that are still in the grouped layout.  Slot j of token t, holding
 * expert e = topk_idx[t][j] of rank r = e / (E / R), has its row at
 *   g(t, j) = slot_pos[send_slot[t][r]][j]
 * (none when topk_idx, send_slot or slot_pos is -1: dropped slots count nothing).  Then
 *   acc[i] = fmaf(topk_weights[t][j], y[g(t, j)][i], acc[i])   over those j ascending, f32 from +0
 *   combined_x[t][i] = bf16(acc[i])                            (nearest, ties to even)
 * In:  y [num_grouped_rows][h] bf16; topk_idx, topk_weights [t][k] as the dispatch took them;
 *      send_slot [t][R] and slot_pos [num_recv_rows][k] as ep_dispatch_grouped (or ep_dispatch and
 *      ep_group_by_expert) wrote them.  num_recv_rows and num_grouped_rows are the rows allocated.
 * Out: combined_x [t][h] bf16 (a token without rows gets zeros).
 * y and combined_x 16-byte, topk_idx 8-byte, the others 4-byte aligned.  One launch.  Limit: fewer
 * than 2^23 KiB pieces in the tokens' rows, each row rounded up (EP_ERR_UNSUPPORTED).
 * dev_status (nullable): EP_DEV_BAD_TOPK_IDX (an id outside [-1, E)), EP_DEV_BAD_SEND_SLOT (a
 * send_slot outside [-1, num_recv_rows) or a slot_pos outside [-1, num_grouped_rows)); such slots
 * are skipped.
 */
ep_status_t ep_combine_grouped(const ep_shape_t *s, const void *y, const int64_t *topk_idx, const float *topk_weights,
                               const int32_t *send_slot, const int32_t *slot_pos, int32_t num_recv_rows,
                               int32_t num_grouped_rows, void *combined_x, int32_t *dev_status, hipStream_t stream);

/*
 * Gradient of ep_combine_grouped.  For every slot with a row g = g(t, j) as there:
 *   grad_y[g][i]              = bf16(topk_weights[t][j] * grad_combined[t][i])   (product in f32)
 *   grad_topk_weights[t][j]   = sum_i y[g][i] * grad_combined[t][i]              (f32)
 * and 0 for grad_topk_weights of the other slots.  Padding rows of the grouped layout, the rows g
 * < min(*num_grouped, num_grouped_rows) with grouped_row[g] < 0, get zeros in grad_y; rows behind
 * *num_grouped are left as they were.
 * In:  grad_combined [t][h] bf16; grouped_row [num_grouped_rows] and num_grouped [1] (device) as
 *      the grouping wrote them; the rest as for ep_combine_grouped.
 * Out: grad_y [num_grouped_rows][h] bf16; grad_topk_weights [t][k] f32, which ep_route_backward
 *      takes as grad_weights.  grad_y may not overlap y.
 * Alignment, limit and dev_status as for ep_combine_grouped.  One launch.
 */
ep_status_t ep_combine_grouped_backward(const ep_shape_t *s, const void *grad_combined, const void *y,
                                        const int64_t *topk_idx, const float *topk_weights, const int32_t *send_slot,
                                        const int32_t *slot_pos, const int32_t *grouped_row,
                                        const int32_t *num_grouped, int32_t num_recv_rows, int32_t num_grouped_rows,
                                        void *grad_y, float *grad_topk_weights, int32_t *dev_status,
                                        hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_EXPERTS_H */
