// ep_experts_api.hip -- the extern "C" entry points declared in ep_experts.h: argument checks on
// the host, then kernel launches on the caller's stream.
#include <limits.h>
#include <math.h>

#include "ep_experts_internal.h"

namespace {

using namespace ep;

bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

ep_status_t from_hip(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ERR_HIP; }

ep_status_t router_checked(const ep_shape_t *s, const ep_router_t *r, int32_t logits_type, int64_t stride) {
    const ep_status_t st = check_shape(s);
    if (st != EP_OK) return st;
    if (r == nullptr) return EP_ERR_INVALID_ARG;
    if (r->score != EP_SCORE_SOFTMAX && r->score != EP_SCORE_SIGMOID) return EP_ERR_INVALID_ARG;
    if (logits_type != EP_LOGITS_F32 && logits_type != EP_LOGITS_BF16) return EP_ERR_INVALID_ARG;
    if (r->num_groups < 1 || s->num_experts % r->num_groups != 0 || r->groups_kept < 1 ||
        r->groups_kept > r->num_groups || (r->group_best != 1 && r->group_best != 2) || !isfinite(r->weight_scale))
        return EP_ERR_INVALID_ARG;
    if (stride < s->num_experts) return EP_ERR_INVALID_ARG;
    if (s->num_experts > kMaxRouteExperts || r->num_groups > kMaxRouteGroups || s->num_tokens > kMaxRouteTokens)
        return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

ep_status_t gemm_checked(const GemmArgs &a) {
    if (a.num_experts < 1 || a.n < 8 || a.n % 8 != 0 || a.k < kScaleBlock || a.k % kScaleBlock != 0 || a.num_rows < 0)
        return EP_ERR_INVALID_ARG;
    if (a.swiglu && a.n % kScaleBlock != 0) return EP_ERR_INVALID_ARG;
    if (a.expert_rows == nullptr && a.num_experts != 1) return EP_ERR_INVALID_ARG;
    if ((int64_t)a.n * (a.swiglu ? 2 : 1) * a.k > INT_MAX || a.k > kMaxGemmK || a.num_experts > kMaxGemmExperts)
        return EP_ERR_UNSUPPORTED;
    if (!gemm_grid_ok(a)) return EP_ERR_UNSUPPORTED;
    if (!aligned(a.expert_rows, 4)) return EP_ERR_INVALID_ARG;
    if (a.num_rows == 0) return EP_OK;
    if (a.x == nullptr || a.x_scales == nullptr || a.w == nullptr || a.w_scales == nullptr || a.out == nullptr ||
        (a.swiglu && a.out_scales == nullptr))
        return EP_ERR_INVALID_ARG;
    if (!aligned(a.x, 16) || !aligned(a.w, 16) || !aligned(a.out, 16) || !aligned(a.x_scales, 4) ||
        !aligned(a.w_scales, 4) || !aligned(a.out_scales, 4))
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

ep_status_t combine_checked(const ep_shape_t *s, const CombineGroupedArgs &a) {
    const ep_status_t st = check_shape(s);
    if (st != EP_OK) return st;
    if (a.num_recv < 0 || a.num_rows < 0) return EP_ERR_INVALID_ARG;
    // a block for each token and KiB of its row, at most, in a grid of 2^31 - 1 threads
    const int64_t pieces = (int64_t)s->num_tokens * ((s->hidden + 511) / 512);
    if (pieces > INT_MAX / 256) return EP_ERR_UNSUPPORTED;
    if (s->num_tokens > 0 && (a.topk_idx == nullptr || a.topk_w == nullptr || a.send_slot == nullptr))
        return EP_ERR_INVALID_ARG;
    if (s->num_tokens > 0 && a.num_recv > 0 && a.slot_pos == nullptr) return EP_ERR_INVALID_ARG;
    if (a.num_rows > 0 && s->num_tokens > 0 && a.y == nullptr) return EP_ERR_INVALID_ARG;
    if (!aligned(a.y, 16) || !aligned(a.grad, 16) || !aligned(a.out, 16) || !aligned(a.topk_idx, 8) ||
        !aligned(a.topk_w, 4) || !aligned(a.send_slot, 4) || !aligned(a.slot_pos, 4) || !aligned(a.grouped_row, 4) ||
        !aligned(a.num_grouped, 4) || !aligned(a.grad_w, 4))
        return EP_ERR_INVALID_ARG;
    return EP_OK;
}

}  // namespace

extern "C" {

ep_status_t ep_route(const ep_shape_t *s, const ep_router_t *r, const void *logits, int32_t logits_type,
                     int64_t logits_stride, const float *bias, const uint8_t *token_mask, int64_t *topk_idx,
                     float *topk_weights, int32_t *dev_status, hipStream_t stream) {
    const ep_status_t st = router_checked(s, r, logits_type, logits_stride);
    if (st != EP_OK) return st;
    if (s->num_tokens == 0) return EP_OK;
    if (logits == nullptr || topk_idx == nullptr || topk_weights == nullptr) return EP_ERR_INVALID_ARG;
    if (!aligned(logits, logits_type == EP_LOGITS_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(topk_idx, 8) ||
        !aligned(topk_weights, 4))
        return EP_ERR_INVALID_ARG;
    RouteArgs a = {};
    a.logits = logits;
    a.stride = logits_stride;
    a.bf16 = logits_type == EP_LOGITS_BF16;
    a.bias = bias;
    a.token_mask = token_mask;
    a.topk_idx = topk_idx;
    a.topk_w = topk_weights;
    a.dev_status = dev_status;
    return from_hip(launch_route(*s, *r, a, stream));
}

ep_status_t ep_route_backward(const ep_shape_t *s, const ep_router_t *r, const void *logits, int32_t logits_type,
                              int64_t logits_stride, const int64_t *topk_idx, const float *grad_weights,
                              void *grad_logits, int64_t grad_stride, int32_t *dev_status, hipStream_t stream) {
    const ep_status_t st = router_checked(s, r, logits_type, logits_stride);
    if (st != EP_OK) return st;
    if (grad_stride < s->num_experts) return EP_ERR_INVALID_ARG;
    if (s->num_tokens == 0) return EP_OK;
    if (logits == nullptr || topk_idx == nullptr || grad_weights == nullptr || grad_logits == nullptr)
        return EP_ERR_INVALID_ARG;
    const uintptr_t width = logits_type == EP_LOGITS_BF16 ? 2 : 4;
    if (!aligned(logits, width) || !aligned(grad_logits, width) || !aligned(topk_idx, 8) || !aligned(grad_weights, 4))
        return EP_ERR_INVALID_ARG;
    RouteBackwardArgs a = {};
    a.logits = logits;
    a.stride = logits_stride;
    a.bf16 = logits_type == EP_LOGITS_BF16;
    a.topk_idx = topk_idx;
    a.grad_w = grad_weights;
    a.grad_logits = grad_logits;
    a.grad_stride = grad_stride;
    a.dev_status = dev_status;
    return from_hip(launch_route_backward(*s, *r, a, stream));
}

ep_status_t ep_expert_gemm_fp8(int32_t num_experts, int32_t n, int32_t k, const void *x, const float *x_scales,
                               const void *w, const float *w_scales, const int32_t *expert_rows, int32_t num_rows,
                               void *out, int32_t *dev_status, hipStream_t stream) {
    GemmArgs a = {};
    a.num_experts = num_experts;
    a.n = n;
    a.k = k;
    a.x = static_cast<const uint8_t *>(x);
    a.x_scales = x_scales;
    a.w = static_cast<const uint8_t *>(w);
    a.w_scales = w_scales;
    a.expert_rows = expert_rows;
    a.num_rows = num_rows;
    a.out = out;
    a.dev_status = dev_status;
    const ep_status_t st = gemm_checked(a);
    if (st != EP_OK) return st;
    return from_hip(launch_expert_gemm(a, stream));
}

ep_status_t ep_expert_gemm_swiglu_fp8(int32_t num_experts, int32_t n, int32_t k, const void *x,
                                      const float *x_scales, const void *w, const float *w_scales,
                                      const int32_t *expert_rows, int32_t num_rows, void *out, float *out_scales,
                                      int32_t *dev_status, hipStream_t stream) {
    GemmArgs a = {};
    a.num_experts = num_experts;
    a.n = n;
    a.k = k;
    a.x = static_cast<const uint8_t *>(x);
    a.x_scales = x_scales;
    a.w = static_cast<const uint8_t *>(w);
    a.w_scales = w_scales;
    a.expert_rows = expert_rows;
    a.num_rows = num_rows;
    a.out = out;
    a.out_scales = out_scales;
    a.dev_status = dev_status;
    a.swiglu = true;
    const ep_status_t st = gemm_checked(a);
    if (st != EP_OK) return st;
    return from_hip(launch_expert_gemm(a, stream));
}

ep_status_t ep_combine_grouped(const ep_shape_t *s, const void *y, const int64_t *topk_idx, const float *topk_weights,
                               const int32_t *send_slot, const int32_t *slot_pos, int32_t num_recv_rows,
                               int32_t num_grouped_rows, void *combined_x, int32_t *dev_status, hipStream_t stream) {
    CombineGroupedArgs a = {};
    a.y = y;
    a.topk_idx = topk_idx;
    a.topk_w = topk_weights;
    a.send_slot = send_slot;
    a.slot_pos = slot_pos;
    a.num_recv = num_recv_rows;
    a.num_rows = num_grouped_rows;
    a.out = combined_x;
    a.dev_status = dev_status;
    const ep_status_t st = combine_checked(s, a);
    if (st != EP_OK || s->num_tokens == 0) return st;
    if (combined_x == nullptr) return EP_ERR_INVALID_ARG;
    return from_hip(launch_combine_grouped(*s, a, stream));
}

ep_status_t ep_combine_grouped_backward(const ep_shape_t *s, const void *grad_combined, const void *y,
                                        const int64_t *topk_idx, const float *topk_weights, const int32_t *send_slot,
                                        const int32_t *slot_pos, const int32_t *grouped_row,
                                        const int32_t *num_grouped, int32_t num_recv_rows, int32_t num_grouped_rows,
                                        void *grad_y, float *grad_topk_weights, int32_t *dev_status,
                                        hipStream_t stream) {
    CombineGroupedArgs a = {};
    a.y = y;
    a.grad = grad_combined;
    a.topk_idx = topk_idx;
    a.topk_w = topk_weights;
    a.send_slot = send_slot;
    a.slot_pos = slot_pos;
    a.grouped_row = grouped_row;
    a.num_grouped = num_grouped;
    a.num_recv = num_recv_rows;
    a.num_rows = num_grouped_rows;
    a.out = grad_y;
    a.grad_w = grad_topk_weights;
    a.dev_status = dev_status;
    const ep_status_t st = combine_checked(s, a);
    if (st != EP_OK) return st;
    if (s->num_tokens > 0 && (grad_combined == nullptr || grad_topk_weights == nullptr)) return EP_ERR_INVALID_ARG;
    if (num_grouped_rows > 0 && (grad_y == nullptr || grouped_row == nullptr || num_grouped == nullptr))
        return EP_ERR_INVALID_ARG;
    return from_hip(launch_combine_grouped_backward(*s, a, stream));
}

}  // extern "C"
