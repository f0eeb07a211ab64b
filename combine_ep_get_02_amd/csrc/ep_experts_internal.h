// ep_experts_internal.h -- private to libep.so: arguments and launchers of the router, the
// experts' products and the grouped combine, and what their kernels share.
#pragma once

#include "ep_experts.h"
#include "ep_internal.h"

namespace ep {

constexpr int kMaxRouteExperts = 2048;
constexpr int kMaxRouteGroups = 64;  // one group per lane of a wave
constexpr int kMaxRouteTokens = 1 << 25;  // a wave each stays within a grid of 2^32 threads
constexpr int kMaxGemmExperts = 16384;
constexpr int kMaxGemmK = 1 << 20;  // a tile's rows are within reach of a 32-bit offset
constexpr int kScaleBlock = 128;  // channels (and weight rows) per scale

struct RouteArgs {
    const void *logits;
    int64_t stride;  // elements between rows
    bool bf16;
    const float *bias;          // may be null
    const uint8_t *token_mask;  // may be null
    int64_t *topk_idx;
    float *topk_w;
    int32_t *dev_status;
};
hipError_t launch_route(const ep_shape_t &s, const ep_router_t &r, const RouteArgs &a, hipStream_t stream);

struct RouteBackwardArgs {
    const void *logits;
    int64_t stride;
    bool bf16;
    const int64_t *topk_idx;
    const float *grad_w;
    void *grad_logits;
    int64_t grad_stride;
    int32_t *dev_status;
};
hipError_t launch_route_backward(const ep_shape_t &s, const ep_router_t &r, const RouteBackwardArgs &a,
                                 hipStream_t stream);

// One product over the grouped rows.  swiglu: w holds 2 n rows an expert and out is E4M3 codes
// with out_scales; otherwise out is bf16.
struct GemmArgs {
    int num_experts, n, k;
    const uint8_t *x;
    const float *x_scales;
    const uint8_t *w;
    const float *w_scales;
    const int32_t *expert_rows;  // null: one expert, all rows
    int num_rows;
    void *out;
    float *out_scales;
    int32_t *dev_status;
    bool swiglu;
};
// False when the launch would need more than 2^31 - 1 threads.
bool gemm_grid_ok(const GemmArgs &a);
hipError_t launch_expert_gemm(const GemmArgs &a, hipStream_t stream);

struct CombineGroupedArgs {
    const void *y;
    const void *grad;  // backward: [t][h] bf16
    const int64_t *topk_idx;
    const float *topk_w;
    const int32_t *send_slot;
    const int32_t *slot_pos;
    const int32_t *grouped_row;  // backward
    const int32_t *num_grouped;  // backward
    int32_t num_recv;
    int32_t num_rows;  // grouped rows allocated
    void *out;         // combined_x, or grad_y (backward)
    float *grad_w;     // backward
    int32_t *dev_status;
};
hipError_t launch_combine_grouped(const ep_shape_t &s, const CombineGroupedArgs &a, hipStream_t stream);
hipError_t launch_combine_grouped_backward(const ep_shape_t &s, const CombineGroupedArgs &a, hipStream_t stream);

// A launch without the triple brackets' pushed and popped configuration: 0.2 us less of the host's 3.7.
template <typename... A>
hipError_t start_kernel(void (*kernel)(A...), int64_t blocks, int threads, hipStream_t stream, A... a) {
    void *args[] = {&a...};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3((unsigned)blocks), dim3(threads),
                                         args, 0, stream);
    if (e != hipSuccess) (void)hipGetLastError();  // it is reported here, and not again by a later call
    return e;
}

// Orders LDS accesses of the wave's own lanes among each other (they are served in order, but
// the compiler does not know that one lane's stores are for another's loads).
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

// Two f32 to a pair of bf16 in one word, nearest, ties to even, NaN kept (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float bf16_low(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_high(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

}  // namespace ep
