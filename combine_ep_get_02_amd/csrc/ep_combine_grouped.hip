// ep_combine_grouped.hip -- the weighted sum of grouped expert outputs in token order, and its
// gradient (gfx950).  Definitions in ep_experts.h.
//
// Both are gathers: the k rows of a token are found through topk_idx -> rank -> send_slot ->
// slot_pos (lane j does slot j), read once with 16-byte loads, and bound by HBM.
#include "ep_experts_internal.h"

namespace ep {
namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

struct Params {
    CombineGroupedArgs a;
    int64_t T, units;  // tokens; 16-byte units of a row
    int E, R, K, segments;
};

// Lane j < K: the grouped row of token t's slot j (-1 without one) and its weight.
__device__ __forceinline__ int find_row(const Params &p, int64_t t, int lane, float *weight, int *bad) {
    int row = -1;
    *weight = 0.0f;
    *bad = 0;
    if (lane < p.K) {
        const int64_t e = p.a.topk_idx[t * p.K + lane];
        *weight = p.a.topk_w[t * p.K + lane];
        if (e < -1 || e >= p.E) {
            *bad = EP_DEV_BAD_TOPK_IDX;
        } else if (e >= 0) {
            const int slot = p.a.send_slot[t * p.R + (int)e / (p.E / p.R)];
            if (slot < -1 || slot >= p.a.num_recv) {
                *bad = EP_DEV_BAD_SEND_SLOT;
            } else if (slot >= 0) {
                row = p.a.slot_pos[(int64_t)slot * p.K + lane];
                if (row < -1 || row >= p.a.num_rows) {
                    *bad = EP_DEV_BAD_SEND_SLOT;
                    row = -1;
                }
            }
        }
    }
    return row;
}

__device__ __forceinline__ void report(const Params &p, int lane, int bad) {
    int bits = 0;
    if (ballot64(bad == EP_DEV_BAD_TOPK_IDX) != 0ull) bits |= EP_DEV_BAD_TOPK_IDX;
    if (ballot64(bad == EP_DEV_BAD_SEND_SLOT) != 0ull) bits |= EP_DEV_BAD_SEND_SLOT;
    if (lane == 0) flag(p.a.dev_status, bits);
}

constexpr int kWaves = 4;

// One wave per (token, segment of 64 * VPL 16-byte units).
template <int VPL>
__global__ __launch_bounds__(kWaves *kWave) void combine_grouped_kernel(Params p) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t w = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (w >= p.T * p.segments) return;  // whole wave leaves together
    const int64_t t = w / p.segments;
    const int seg = (int)(w - t * p.segments);
    float weight;
    int bad;
    const int row = find_row(p, t, lane, &weight, &bad);
    if (seg == 0) report(p, lane, bad);
    const int64_t c0 = (int64_t)seg * VPL * kWave + lane;
    const u32x4 *y = static_cast<const u32x4 *>(p.a.y);

    float acc[VPL][8];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[i][k] = 0.0f;
    for (uint64_t todo = ballot64(row >= 0); todo != 0ull; todo &= todo - 1ull) {
        const int j = __builtin_ctzll(todo);
        const float wj = readlanef(weight, j);
        const u32x4 *src = y + (int64_t)readlane32(row, j) * p.units + c0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            if (c0 + i * kWave < p.units) {
                const u32x4 v = __builtin_nontemporal_load(src + i * kWave);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[i][2 * k] = __builtin_fmaf(wj, bf16_low(v[k]), acc[i][2 * k]);
                    acc[i][2 * k + 1] = __builtin_fmaf(wj, bf16_high(v[k]), acc[i][2 * k + 1]);
                }
            }
        }
    }
    u32x4 *dst = static_cast<u32x4 *>(p.a.out) + t * p.units + c0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        u32x4 o;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = pack_bf16(acc[i][2 * k], acc[i][2 * k + 1]);
        if (c0 + i * kWave < p.units) __builtin_nontemporal_store(o, dst + i * kWave);
    }
}

// One block per token: the token's gradient row is scaled into each of its grouped rows, and its
// product with that row's output summed over the block.  After its token a block zeroes the
// padding rows among grouped rows blockIdx.x, blockIdx.x + gridDim.x, ...
__global__ __launch_bounds__(kWaves *kWave) void combine_grouped_backward_kernel(Params p) {
    __shared__ float s_dot[kMaxTopk][kWaves];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x >> 6;
    const int64_t t = blockIdx.x;
    const u32x4 *y = static_cast<const u32x4 *>(p.a.y);
    u32x4 *gy = static_cast<u32x4 *>(p.a.out);
    if (t < p.T) {
        float weight;
        int bad;
        const int row = find_row(p, t, lane, &weight, &bad);
        if (wave == 0) report(p, lane, bad);
        const u32x4 *grad = static_cast<const u32x4 *>(p.a.grad) + t * p.units;
        const uint64_t there = ballot64(row >= 0);
        for (uint64_t todo = there; todo != 0ull; todo &= todo - 1ull) {
            const int j = __builtin_ctzll(todo);
            const float wj = readlanef(weight, j);
            const int64_t at = (int64_t)readlane32(row, j) * p.units;
            float dot = 0.0f;
            for (int64_t c = threadIdx.x; c < p.units; c += kWaves * kWave) {
                const u32x4 v = __builtin_nontemporal_load(y + at + c);
                const u32x4 g = grad[c];
                u32x4 o;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    dot = __builtin_fmaf(bf16_low(v[k]), bf16_low(g[k]), dot);
                    dot = __builtin_fmaf(bf16_high(v[k]), bf16_high(g[k]), dot);
                    o[k] = pack_bf16(wj * bf16_low(g[k]), wj * bf16_high(g[k]));
                }
                __builtin_nontemporal_store(o, gy + at + c);
            }
            for (int s = 1; s < kWave; s <<= 1) dot += __shfl_xor(dot, s);
            if (lane == 0) s_dot[j][wave] = dot;
        }
        __syncthreads();
        if (wave == 0 && lane < p.K) {
            float dot = 0.0f;
            if ((there >> lane) & 1ull)
                for (int i = 0; i < kWaves; ++i) dot += s_dot[lane][i];
            p.a.grad_w[t * p.K + lane] = dot;
        }
    }
    // padding rows: each wave looks at 64 of the block's rows at a time
    int64_t n = p.a.num_rows;
    if (n > 0) n = *p.a.num_grouped < n ? *p.a.num_grouped : n;
    const u32x4 zero = {0u, 0u, 0u, 0u};
    for (int64_t first = (int64_t)wave * kWave; blockIdx.x + first * gridDim.x < n; first += kWaves * kWave) {
        const int64_t g = blockIdx.x + (first + lane) * gridDim.x;
        uint64_t todo = ballot64(g < n && p.a.grouped_row[g] < 0);
        for (; todo != 0ull; todo &= todo - 1ull) {
            const int64_t r = blockIdx.x + (first + __builtin_ctzll(todo)) * gridDim.x;
            for (int64_t c = lane; c < p.units; c += kWave) gy[r * p.units + c] = zero;
        }
    }
}

Params params(const ep_shape_t &s, const CombineGroupedArgs &a) {
    Params p;
    p.a = a;
    p.T = s.num_tokens;
    p.units = s.hidden / 8;
    p.E = s.num_experts;
    p.R = s.num_ranks;
    p.K = s.num_topk;
    p.segments = 1;
    return p;
}

}  // namespace

hipError_t launch_combine_grouped(const ep_shape_t &s, const CombineGroupedArgs &a, hipStream_t stream) {
    if (s.num_tokens == 0) return hipSuccess;
    Params p = params(s, a);
    constexpr int VPL = 2;
    p.segments = (int)((p.units + VPL * kWave - 1) / (VPL * kWave));
    const int64_t blocks = (p.T * p.segments + kWaves - 1) / kWaves;
    hipLaunchKernelGGL((combine_grouped_kernel<VPL>), dim3((unsigned)blocks), dim3(kWaves * kWave), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_combine_grouped_backward(const ep_shape_t &s, const CombineGroupedArgs &a, hipStream_t stream) {
    const Params p = params(s, a);
    // a block per token, and enough of them for the padding of a batch of few tokens
    int64_t blocks = a.num_rows / 16 < 1024 ? a.num_rows / 16 + 1 : 1024;
    if (p.T > blocks) blocks = p.T;
    if (p.T == 0 && a.num_rows == 0) return hipSuccess;
    hipLaunchKernelGGL(combine_grouped_backward_kernel, dim3((unsigned)blocks), dim3(kWaves * kWave), 0, stream, p);
    return hipGetLastError();
}

}  // namespace ep
