// ep_route.hip -- the router: a token's scores, the experts chosen from them and their weights, and
// the gradient of the weights (gfx950).  Definitions in ep_experts.h.
//
// One wave per token.  Lane i holds the VPL consecutive experts from i * VPL, so the lowest lane
// with the largest value, then the lowest element in it, is the lowest expert: ties need no index.
// Choices are compared in binary64: a last-bit difference of a 32-bit exp would otherwise decide
// which of two nearly equal experts a token goes to.
#include "ep_experts_internal.h"

namespace ep {
namespace {

constexpr int kRouteWaves = 4;  // waves (tokens) per block

struct RouteParams {
    RouteArgs a;
    int64_t T;
    int E, K, G, kept, best, group_size;
    bool sigmoid, renorm;
    float scale;
};

struct RouteBackwardParams {
    RouteBackwardArgs a;
    int64_t T;
    int E, K;
    bool sigmoid, renorm;
    float scale;
};

template <bool BF16>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
    if constexpr (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
    return static_cast<const float *>(p)[i];
}

__device__ __forceinline__ double shfl_xor_f64(double v, int s) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __shfl_xor((int)(uint32_t)u, s), hi = __shfl_xor((int)(uint32_t)(u >> 32), s);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ double readlane_f64(double v, int src) {
    return __builtin_bit_cast(double, readlane64(__builtin_bit_cast(uint64_t, v), src));
}

__device__ __forceinline__ double wave_max_f64(double v) {
    for (int s = 1; s < kWave; s <<= 1) {
        const double o = shfl_xor_f64(v, s);
        v = o > v ? o : v;
    }
    return v;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
    for (int s = 1; s < kWave; s <<= 1) v += shfl_xor_f64(v, s);
    return v;
}

__device__ __forceinline__ float wave_max_f32(float v) {
    for (int s = 1; s < kWave; s <<= 1) v = fmaxf(v, __shfl_xor(v, s));
    return v;
}

__device__ __forceinline__ float wave_sum_f32(float v) {
    for (int s = 1; s < kWave; s <<= 1) v += __shfl_xor(v, s);
    return v;
}

// NaN and +inf: not a logit (or bias) the router can use.
__device__ __forceinline__ bool unusable(float v) { return !(v < INFINITY); }

template <int VPL, bool BF16>
__global__ __launch_bounds__(kRouteWaves *kWave) void route_kernel(RouteParams p) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
    if (t >= p.T) return;  // whole wave leaves together
    int64_t *idx_out = p.a.topk_idx + t * p.K;
    float *w_out = p.a.topk_w + t * p.K;
    if (p.a.token_mask != nullptr && p.a.token_mask[t] == 0) {
        if (lane < p.K) {
            idx_out[lane] = -1;
            w_out[lane] = 0.0f;
        }
        return;
    }
    const double none = -INFINITY;
    const int e0 = lane * VPL;
    float logit[VPL];
    bool bad = false;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        float l = -INFINITY;
        if (e0 + i < p.E) l = load_logit<BF16>(p.a.logits, t * p.a.stride + e0 + i);
        if (unusable(l)) {
            bad = true;
            l = -INFINITY;
        }
        logit[i] = l;
        top = fmaxf(top, l);
    }
    top = wave_max_f32(top);

    // choice[i]: c_e; key[i]: what orders the experts (c_e, or the logit when there is no bias)
    double choice[VPL], sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        choice[i] = 0.0;
        if (logit[i] > -INFINITY) {
            const double l = logit[i];
            choice[i] = p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top);
        }
        sum += choice[i];
    }
    if (!p.sigmoid) {
        sum = wave_sum_f64(sum);
#pragma unroll
        for (int i = 0; i < VPL; ++i) choice[i] /= sum;
    }
    double key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        key[i] = logit[i];
        if (p.a.bias != nullptr) {
            float b = e0 + i < p.E ? p.a.bias[e0 + i] : -INFINITY;
            if (unusable(b)) {
                bad = true;
                b = -INFINITY;
            }
            if (b == -INFINITY) key[i] = none;
            choice[i] += (double)b;
            if (key[i] > none) key[i] = choice[i];
        }
    }
    if (ballot64(bad) != 0ull && lane == 0) flag(p.a.dev_status, EP_DEV_BAD_LOGIT);

    if (p.G > 1) {
        // lane g: rating of group g
        double rating = none;
        for (int g = 0; g < p.G; ++g) {
            const int lo = g * p.group_size, hi = lo + p.group_size;
            const bool by_logit = p.best == 1 && p.a.bias == nullptr;
            double a = none, b = none;  // the two largest of this lane's part of the group
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (e0 + i >= lo && e0 + i < hi && key[i] > none) {
                    const double v = by_logit ? key[i] : choice[i];
                    if (v > a) {
                        b = a;
                        a = v;
                    } else if (v > b) {
                        b = v;
                    }
                }
            }
            for (int s = 1; s < kWave; s <<= 1) {
                const double oa = shfl_xor_f64(a, s), ob = shfl_xor_f64(b, s);
                const double low = a < oa ? a : oa;
                a = a > oa ? a : oa;
                b = b > ob ? b : ob;
                b = b > low ? b : low;
            }
            const double r = p.best == 2 && b > none ? a + b : a;
            if (lane == g) rating = r;
        }
        int ahead = 0;  // groups rated above lane's group
        for (int g = 0; g < p.G; ++g) {
            const double o = readlane_f64(rating, g);
            ahead += o > rating || (o == rating && g < lane);
        }
        const uint64_t keep = ballot64(lane < p.G && ahead < p.kept);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int g = (e0 + i) / p.group_size;
            if (g >= kWave || ((keep >> g) & 1ull) == 0ull) key[i] = none;
        }
    }

    // num_topk rounds: the largest key left, lowest expert first; lane j keeps round j's expert
    int chosen = -1;
    for (int j = 0; j < p.K; ++j) {
        double m = none;
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = key[i] > m ? key[i] : m;
        const double best = wave_max_f64(m);
        if (!(best > none)) break;
        const int owner = __builtin_ctzll(ballot64(m == best));
        int e = -1;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
            if (key[i] == best) e = i;
        e = readlane32(e, owner);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane == owner && i == e) key[i] = none;
        if (lane == j) chosen = owner * VPL + e;
    }

    double s = 0.0;
    if (chosen >= 0) {
        const double l = load_logit<BF16>(p.a.logits, t * p.a.stride + chosen);
        s = p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) / sum;
    }
    double w = s * (double)p.scale;
    if (p.renorm) {
        const double all = wave_sum_f64(s);
        w = all > 0.0 ? w / all : 0.0;
    }
    if (lane < p.K) {
        idx_out[lane] = chosen;
        w_out[lane] = (float)w;
    }
}

template <int VPL, bool BF16>
__global__ __launch_bounds__(kRouteWaves *kWave) void route_backward_kernel(RouteBackwardParams p) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6);
    if (t >= p.T) return;  // whole wave leaves together
    const int e0 = lane * VPL;
    float logit[VPL];
    bool bad = false;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        float l = -INFINITY;
        if (e0 + i < p.E) l = load_logit<BF16>(p.a.logits, t * p.a.stride + e0 + i);
        if (unusable(l)) {
            bad = true;
            l = -INFINITY;
        }
        logit[i] = l;
        top = fmaxf(top, l);
    }
    top = wave_max_f32(top);
    float score[VPL], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        score[i] = 0.0f;
        if (logit[i] > -INFINITY) score[i] = p.sigmoid ? 1.0f / (1.0f + expf(-logit[i])) : expf(logit[i] - top);
        sum += score[i];
    }
    if (!p.sigmoid) {
        sum = wave_sum_f32(sum);
#pragma unroll
        for (int i = 0; i < VPL; ++i) score[i] = sum > 0.0f ? score[i] / sum : 0.0f;
    }

    // lane j: slot j's expert, its score and the gradient of that score, in 64 bits: the sums over
    // the slots cancel
    int64_t id = -1;
    double s = 0.0, g = 0.0;
    bool bad_id = false;
    if (lane < p.K) {
        id = p.a.topk_idx[t * p.K + lane];
        if (id < -1 || id >= p.E) {
            bad_id = true;
            id = -1;
        }
        if (id >= 0) {
            const float l = load_logit<BF16>(p.a.logits, t * p.a.stride + id);
            if (l > -INFINITY && !unusable(l))
                s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)top) / (double)sum;
            g = p.a.grad_w[t * p.K + lane];
        }
    }
    if (ballot64(bad) != 0ull && lane == 0) flag(p.a.dev_status, EP_DEV_BAD_LOGIT);
    if (ballot64(bad_id) != 0ull && lane == 0) flag(p.a.dev_status, EP_DEV_BAD_TOPK_IDX);
    double ds = g * (double)p.scale;
    if (p.renorm) {
        const double all = wave_sum_f64(s), gs = wave_sum_f64(id >= 0 ? g * s : 0.0);
        ds = id >= 0 && all > 0.0 ? (double)p.scale * (g - gs / all) / all : 0.0;
    }
    const float slot = (float)ds;
    const float mean = p.sigmoid ? 0.0f : (float)wave_sum_f64(id >= 0 ? ds * s : 0.0);

    float d[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = 0.0f;
    for (int j = 0; j < p.K; ++j) {
        const int e = readlane32((int)id, j);
        const float v = readlanef(slot, j);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (e == e0 + i) d[i] += v;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if (e0 + i >= p.E) continue;
        float v = 0.0f;
        if (logit[i] > -INFINITY) {
            // 1 - s as its own sigmoid: it does not cancel where s is near 1
            if (p.sigmoid)
                v = d[i] * score[i] * (1.0f / (1.0f + expf(logit[i])));
            else
                v = score[i] * (d[i] - mean);
        }
        const int64_t at = t * p.a.grad_stride + e0 + i;
        if constexpr (BF16)
            static_cast<uint16_t *>(p.a.grad_logits)[at] = (uint16_t)pack_bf16(v, 0.0f);
        else
            static_cast<float *>(p.a.grad_logits)[at] = v;
    }
}

template <int VPL, bool BF16>
void start(const RouteParams &p, hipStream_t stream) {
    const unsigned blocks = (unsigned)((p.T + kRouteWaves - 1) / kRouteWaves);
    hipLaunchKernelGGL((route_kernel<VPL, BF16>), dim3(blocks), dim3(kRouteWaves * kWave), 0, stream, p);
}
template <int VPL, bool BF16>
void start(const RouteBackwardParams &p, hipStream_t stream) {
    const unsigned blocks = (unsigned)((p.T + kRouteWaves - 1) / kRouteWaves);
    hipLaunchKernelGGL((route_backward_kernel<VPL, BF16>), dim3(blocks), dim3(kRouteWaves * kWave), 0, stream, p);
}

// The fewest experts a lane that hold E.
template <typename P>
hipError_t start_sized(const P &p, hipStream_t stream) {
#define EP_ROUTE_CASE(V)                   \
    if (p.E <= V * kWave) {                \
        if (p.a.bf16)                      \
            start<V, true>(p, stream);     \
        else                               \
            start<V, false>(p, stream);    \
        return hipGetLastError();          \
    }
    EP_ROUTE_CASE(1)
    EP_ROUTE_CASE(2)
    EP_ROUTE_CASE(4)
    EP_ROUTE_CASE(8)
    EP_ROUTE_CASE(16)
    EP_ROUTE_CASE(32)
#undef EP_ROUTE_CASE
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_route(const ep_shape_t &s, const ep_router_t &r, const RouteArgs &a, hipStream_t stream) {
    if (s.num_tokens == 0) return hipSuccess;
    RouteParams p;
    p.a = a;
    p.T = s.num_tokens;
    p.E = s.num_experts;
    p.K = s.num_topk;
    p.G = r.num_groups;
    p.kept = r.groups_kept;
    p.best = r.group_best;
    p.group_size = s.num_experts / r.num_groups;
    p.sigmoid = r.score == EP_SCORE_SIGMOID;
    p.renorm = r.renormalize != 0;
    p.scale = r.weight_scale;
    return start_sized(p, stream);
}

hipError_t launch_route_backward(const ep_shape_t &s, const ep_router_t &r, const RouteBackwardArgs &a,
                                 hipStream_t stream) {
    if (s.num_tokens == 0) return hipSuccess;
    RouteBackwardParams p;
    p.a = a;
    p.T = s.num_tokens;
    p.E = s.num_experts;
    p.K = s.num_topk;
    p.sigmoid = r.score == EP_SCORE_SIGMOID;
    p.renorm = r.renormalize != 0;
    p.scale = r.weight_scale;
    return start_sized(p, stream);
}

}  // namespace ep
