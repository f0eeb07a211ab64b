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
    int E, R, K;
    int64_t segments;  // waves of a token's row
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

// One wave per (token, segment of 64 16-byte units).  Up to kBatch rows' segments are loaded before
// the first is used: a row at a time, a wave would wait out the memory's latency k times (prefill,
// 4096 tokens of 8 rows of 7168: 87-93 us with 1 to 4 units a lane and batches of 2 to 8 alike, 5.7 to
// 6.1 TB/s; 128 tokens: 4.9 us, a launch included).
constexpr int kBatch = 8;
__global__ __launch_bounds__(kWaves *kWave) void combine_grouped_kernel(Params p) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t w = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (w >= p.T * p.segments) return;  // whole wave leaves together
    const int64_t t = w / p.segments;
    const int64_t c = (w - t * p.segments) * kWave + lane;
    float weight;
    int bad;
    const int row = find_row(p, t, lane, &weight, &bad);
    if (w == t * p.segments) report(p, lane, bad);
    const u32x4 *y = static_cast<const u32x4 *>(p.a.y) + c;
    const bool inside = c < p.units;

    float acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
    uint64_t todo = ballot64(row >= 0);
    while (todo != 0ull) {
        u32x4 v[kBatch];
        float wj[kBatch];
        int n = 0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (todo == 0ull) break;
            const int j = __builtin_ctzll(todo);
            todo &= todo - 1ull;
            wj[u] = readlanef(weight, j);
            const u32x4 *src = y + (int64_t)readlane32(row, j) * p.units;
            if (inside) v[u] = __builtin_nontemporal_load(src);
            n = u + 1;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (u >= n) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[2 * k] = __builtin_fmaf(wj[u], bf16_low(v[u][k]), acc[2 * k]);
                acc[2 * k + 1] = __builtin_fmaf(wj[u], bf16_high(v[u][k]), acc[2 * k + 1]);
            }
        }
    }
    u32x4 o;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = pack_bf16(acc[2 * k], acc[2 * k + 1]);
    if (inside) __builtin_nontemporal_store(o, static_cast<u32x4 *>(p.a.out) + t * p.units + c);
}

// The padding rows among grouped rows blockIdx.x, blockIdx.x + gridDim.x, ... get zeros; each wave
// looks at 64 of the block's rows at a time.
template <int WAVES>
__device__ __forceinline__ void zero_padding(const Params &p) {
    const int lane = threadIdx.x & (kWave - 1);
    u32x4 *gy = static_cast<u32x4 *>(p.a.out);
    int64_t n = p.a.num_rows;
    if (n > 0) n = *p.a.num_grouped < n ? *p.a.num_grouped : n;
    const u32x4 zero = {0u, 0u, 0u, 0u};
    for (int64_t first = (threadIdx.x >> 6) * kWave; blockIdx.x + first * gridDim.x < n; first += WAVES * kWave) {
        const int64_t g = blockIdx.x + (first + lane) * gridDim.x;
        uint64_t todo = ballot64(g < n && p.a.grouped_row[g] < 0);
        for (; todo != 0ull; todo &= todo - 1ull) {
            const int64_t r = blockIdx.x + (first + __builtin_ctzll(todo)) * gridDim.x;
            for (int64_t c = lane; c < p.units; c += kWave) __builtin_nontemporal_store(zero, gy + r * p.units + c);
        }
    }
}

// One block per token: the token's gradient row is scaled into each of its grouped rows, and its
// product with that row's output summed over the block.  The gradient row stays in registers, UPT
// 16-byte units a thread (rows of up to 64 WAVES UPT units; longer ones in turns), and the next row's
// outputs are loaded while one is worked on.  Bound by HBM: 16384 tokens of 6 rows of 4096 take 327 us for 1.75
// GB, 5.3 TB/s; 1000 tokens of 8 rows of 7168 with padding 48 us.
template <int WAVES, int UPT>
__global__ __launch_bounds__(WAVES *kWave) void combine_grouped_backward_kernel(Params p) {
    __shared__ float s_dot[kMaxTopk][WAVES];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x >> 6;
    const int64_t t = blockIdx.x;
    if (t < p.T) {
        float weight;
        int bad;
        const int row = find_row(p, t, lane, &weight, &bad);
        if (wave == 0) report(p, lane, bad);
        const uint64_t there = ballot64(row >= 0);
        float total = 0.0f;  // lane j: of slot j, this wave's part
        for (int64_t from = 0; from < p.units; from += UPT * WAVES * kWave) {
            const int64_t c0 = from + threadIdx.x;
            const u32x4 *grad = static_cast<const u32x4 *>(p.a.grad) + t * p.units + c0;
            const u32x4 *y = static_cast<const u32x4 *>(p.a.y) + c0;
            u32x4 *gy = static_cast<u32x4 *>(p.a.out) + c0;
            u32x4 g[UPT], v[UPT], next[UPT];
            const u32x4 zero = {0u, 0u, 0u, 0u};
            auto load = [&](u32x4(&to)[UPT], const u32x4 *src) {
#pragma unroll
                for (int i = 0; i < UPT; ++i) {
                    to[i] = zero;
                    if (c0 + i * WAVES * kWave < p.units) to[i] = __builtin_nontemporal_load(src + i * WAVES * kWave);
                }
            };
            load(g, grad);
            uint64_t todo = there;
            if (todo != 0ull) load(next, y + (int64_t)readlane32(row, __builtin_ctzll(todo)) * p.units);
            while (todo != 0ull) {
                const int j = __builtin_ctzll(todo);
                todo &= todo - 1ull;
#pragma unroll
                for (int i = 0; i < UPT; ++i) v[i] = next[i];
                if (todo != 0ull) load(next, y + (int64_t)readlane32(row, __builtin_ctzll(todo)) * p.units);
                const float wj = readlanef(weight, j);
                u32x4 *dst = gy + (int64_t)readlane32(row, j) * p.units;
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < UPT; ++i) {
                    u32x4 o;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        dot = __builtin_fmaf(bf16_low(v[i][k]), bf16_low(g[i][k]), dot);
                        dot = __builtin_fmaf(bf16_high(v[i][k]), bf16_high(g[i][k]), dot);
                        o[k] = pack_bf16(wj * bf16_low(g[i][k]), wj * bf16_high(g[i][k]));
                    }
                    if (c0 + i * WAVES * kWave < p.units) __builtin_nontemporal_store(o, dst + i * WAVES * kWave);
                }
                for (int s = 1; s < kWave; s <<= 1) dot += __shfl_xor(dot, s);
                if (lane == j) total += dot;
            }
        }
        if (lane < p.K) s_dot[lane][wave] = total;
        __syncthreads();
        if (wave == 0 && lane < p.K) {
            float dot = 0.0f;
            for (int i = 0; i < WAVES; ++i) dot += s_dot[lane][i];
            p.a.grad_w[t * p.K + lane] = dot;
        }
    }
    zero_padding<WAVES>(p);
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
    p.segments = (p.units + kWave - 1) / kWave;
    const int64_t blocks = (p.T * p.segments + kWaves - 1) / kWaves;
    return start_kernel(combine_grouped_kernel, blocks, kWaves * kWave, stream, p);
}

hipError_t launch_combine_grouped_backward(const ep_shape_t &s, const CombineGroupedArgs &a, hipStream_t stream) {
    const Params p = params(s, a);
    // a block per token, and enough of them for the padding of a batch of few tokens
    int64_t blocks = a.num_rows / 16 < 1024 ? a.num_rows / 16 + 1 : 1024;
    if (p.T > blocks) blocks = p.T;
    if (p.T == 0 && a.num_rows == 0) return hipSuccess;
    // rows up to 4 KiB in one turn of four waves; wider ones take 8 waves of two units (16 KiB a turn).  16384 tokens of
    // 6 rows of 4096 / 1000 of 8 rows of 7168 with padding, us in a graph: 323 / 48; 4 waves of two units 330 / 51, of
    // four 325 / 48, 16 waves of one 338 / 49
    if (p.units <= 4 * kWave) return start_kernel(combine_grouped_backward_kernel<4, 1>, blocks, 4 * kWave, stream, p);
    return start_kernel(combine_grouped_backward_kernel<8, 2>, blocks, 8 * kWave, stream, p);
}

}  // namespace ep
