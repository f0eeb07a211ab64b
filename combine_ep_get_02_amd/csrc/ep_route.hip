// ep_route.hip -- the router: a token's scores, the experts chosen from them and their weights, and
// the gradient of the weights (gfx950).  Definitions in ep_experts.h.
//
// A token is 64 lanes or, where there are many tokens and few experts, 32 or 16 (a round of the selection
// then costs its cross-lane steps once for two or four tokens of a wave).  Lane i of a token holds
// the VPL consecutive experts from i * VPL, so the lowest lane with the largest value, then the
// lowest element in it, is the lowest expert: ties need no index.
//
// Choices compare as in binary64 -- a last-bit difference of a 32-bit exp must not decide which of
// two nearly equal experts a token goes to -- but are formed in f32 first.  With no bias the logits
// themselves order the experts, and f32 is exact.  Otherwise f32 choices are off by a known part
// of their size.  Where two neighbours in the order found are no further apart than that, the order
// is followed down to a wider step, and the experts above it are ordered anew in binary64; where the
// last group kept and the best one dropped are, the groups are rated in binary64.
#include <limits.h>

#include "ep_experts_internal.h"

namespace ep {
namespace {

constexpr int kRouteWaves = 4;  // waves per block
// From this many tokens on they share waves.  Few tokens are bound by the latency of one wave's steps, which
// more experts a lane lengthen; many by the vector instructions of all.  8 slots, router (softmax) / its
// gradient (softmax, not renormalised) with 64, 32 and 16 lanes, us:
//   tokens                    2048                          4096                          16384
//   64 experts                4.6/3.5  4.6/3.7  4.8/4.0     5.5/4.5  4.9/4.0  4.8/4.1     13.0/10.6  9.2/7.7  6.5/6.3
//   128 experts               4.8/4.0  4.9/4.1  5.5/4.8     6.0/5.4  5.4/4.5  5.6/5.2     14.5/13.6  10.4/9.9  8.0/9.1
//   256 experts in 8 groups   7.9/4.6  9.1/5.1  17.7/8.1    11/6.4   10/5.9   18/8.7      29/18.4    25/15.4   30/17.3
// (512 experts in 8 groups, 16384 tokens, router with 64 and 32 lanes: 40 and 41.)
constexpr int64_t kManyTokens = 4096;

struct RouteParams {
    RouteArgs a;
    int64_t T;
    int E, K, G, kept, best, group_size;
    int group_lanes;  // lanes of a token that share a group: a power of two, of all lanes over G
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

__device__ __forceinline__ double shfl_f64(double v, int from) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __shfl((int)(uint32_t)u, from), hi = __shfl((int)(uint32_t)(u >> 32), from);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// VPL values of a row from element i on, `left` of them there (the others are left as they are).  Where
// all are, in words of up to 16 bytes, which need not lie on boundaries of more than 4.
template <int VPL>
__device__ __forceinline__ void load_values(const float *p, int64_t i, int left, float (&out)[VPL]) {
    constexpr int W = VPL < 4 ? VPL : 4;
    typedef float vec __attribute__((ext_vector_type(W), aligned(4)));
    if (left >= VPL) {
#pragma unroll
        for (int k = 0; k < VPL; k += W) {
            const vec v = *reinterpret_cast<const vec *>(p + i + k);
#pragma unroll
            for (int u = 0; u < W; ++u) out[k + u] = v[u];
        }
    } else {
#pragma unroll
        for (int k = 0; k < VPL; ++k)
            if (k < left) out[k] = p[i + k];
    }
}

__device__ __forceinline__ bool on_words(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

template <int VPL, bool BF16>
__device__ __forceinline__ void load_logits(const void *p, int64_t i, int left, float (&out)[VPL]) {
    if constexpr (!BF16) {
        load_values<VPL>(static_cast<const float *>(p), i, left, out);
    } else {
        constexpr int W = VPL < 2 ? 1 : VPL < 8 ? VPL / 2 : 4;
        typedef uint32_t vec __attribute__((ext_vector_type(W), aligned(4)));
        const uint16_t *src = static_cast<const uint16_t *>(p) + i;
        if (VPL > 1 && left >= VPL && on_words(src)) {
#pragma unroll
            for (int k = 0; k < VPL; k += 2 * W) {
                const vec v = *reinterpret_cast<const vec *>(src + k);
#pragma unroll
                for (int u = 0; u < 2 * W && k + u < VPL; ++u) out[k + u] = u % 2 == 0 ? bf16_low(v[u / 2]) : bf16_high(v[u / 2]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < VPL; ++k)
                if (k < left) out[k] = __uint_as_float((uint32_t)src[k] << 16);
        }
    }
}

template <int VPL, bool BF16>
__device__ __forceinline__ void store_logits(void *p, int64_t i, int left, const float (&v)[VPL]) {
    if (left < VPL || (BF16 && !on_words(static_cast<uint16_t *>(p) + i))) {
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            if (k >= left) continue;
            if constexpr (BF16)
                static_cast<uint16_t *>(p)[i + k] = (uint16_t)pack_bf16(v[k], 0.0f);
            else
                static_cast<float *>(p)[i + k] = v[k];
        }
    } else if constexpr (BF16 && VPL == 1) {
        static_cast<uint16_t *>(p)[i] = (uint16_t)pack_bf16(v[0], 0.0f);
    } else if constexpr (BF16) {
        constexpr int W = VPL < 8 ? VPL / 2 : 4;
        typedef uint32_t vec __attribute__((ext_vector_type(W), aligned(4)));
#pragma unroll
        for (int k = 0; k < VPL; k += 2 * W) {
            vec w;
#pragma unroll
            for (int u = 0; u < W; ++u) w[u] = pack_bf16(v[k + 2 * u], v[k + 2 * u + 1]);
            *reinterpret_cast<vec *>(static_cast<uint16_t *>(p) + i + k) = w;
        }
    } else {
        constexpr int W = VPL < 4 ? VPL : 4;
        typedef float vec __attribute__((ext_vector_type(W), aligned(4)));
#pragma unroll
        for (int k = 0; k < VPL; k += W) {
            vec w;
#pragma unroll
            for (int u = 0; u < W; ++u) w[u] = v[k + u];
            *reinterpret_cast<vec *>(static_cast<float *>(p) + i + k) = w;
        }
    }
}

// NaN and +inf: not a logit (or bias) the router can use.
__device__ __forceinline__ bool unusable(float v) { return !(v < INFINITY); }

// How far apart two f32 choices have to be for their order to be sure: kSlack of the larger one's size
// and kSigmoidSlack, or kSoftmaxSlack of the token's largest score.  With u = 2^-24: an exponential is off by
// (|argument| + 2) u of it at most.  A sigmoid's argument -l is exact, and its exponential weighs (1 - s) in
// the score: s (1 - s) (|l| + 2) u < 0.6 u.  Its sum and its quotient add s u each, so it is off by under
// 2.6 u; adding the bias by u of the choice.  The argument l - max of a softmax leaves its exponential under
// 2 u of 1 off; it divides by a sum whose terms are off by the same and whose 38 additions at most by u each:
// under 60 u of the largest score.  Twice that for two sides, and half as much again to spare.
constexpr float kSlack = 4 * 0x1p-24f, kSigmoidSlack = 8 * 0x1p-24f, kSoftmaxSlack = 180 * 0x1p-24f;

// f32 to an integer that orders as it does (+0 and -0 alike); kNone is below all of them.
constexpr int kNone = INT_MIN;
__device__ __forceinline__ int order_of(float v) {
    const int b = __float_as_int(v + 0.0f);
    return b ^ ((b >> 31) & INT_MAX);
}
__device__ __forceinline__ float value_of(int o) { return __int_as_float(o ^ ((o >> 31) & INT_MAX)); }

// Largest value over a token's LPT lanes, for all of them.
template <int LPT>
__device__ __forceinline__ int token_max(int v) {
    if constexpr (LPT == kWave) {
#define EP_MAX_STEP(ctrl, rows) \
    { const int o = __builtin_amdgcn_update_dpp(v, v, ctrl, rows, 0xf, false); v = o > v ? o : v; }
        EP_MAX_STEP(0x111, 0xf)  // row_shr:1
        EP_MAX_STEP(0x112, 0xf)  // row_shr:2
        EP_MAX_STEP(0x114, 0xf)  // row_shr:4
        EP_MAX_STEP(0x118, 0xf)  // row_shr:8
        EP_MAX_STEP(0x142, 0xa)  // row_bcast:15 into rows 1, 3
        EP_MAX_STEP(0x143, 0xc)  // row_bcast:31 into rows 2, 3
#undef EP_MAX_STEP
        return readlane32(v, kWave - 1);
    } else {
        static_assert(LPT == 16 || LPT == 32, "one row of 16 lanes or two");
        int o = (int)lane_xor<1>((uint32_t)v);
        v = o > v ? o : v;
        o = (int)lane_xor<2>((uint32_t)v);
        v = o > v ? o : v;
        o = (int)lane_xor<4>((uint32_t)v);
        v = o > v ? o : v;
        o = (int)lane_xor<8>((uint32_t)v);
        v = o > v ? o : v;
        if constexpr (LPT == 32) {
            o = (int)lane_xor<16>((uint32_t)v);
            v = o > v ? o : v;
        }
        return v;
    }
}

// v of lane ^ S, for S below 16 without a trip through LDS.
template <int S>
__device__ __forceinline__ float of_lane_xor(float v) {
    return __uint_as_float(lane_xor<S>(__float_as_uint(v)));
}
template <int S>
__device__ __forceinline__ double of_lane_xor(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, ((uint64_t)lane_xor<S>((uint32_t)(u >> 32)) << 32) | lane_xor<S>((uint32_t)u));
}
__device__ __forceinline__ float of_lane(float v, int l) { return readlanef(v, l); }
__device__ __forceinline__ double of_lane(double v, int l) {
    return __builtin_bit_cast(double, readlane64(__builtin_bit_cast(uint64_t, v), l));
}

// Sum over a token's lanes, in one order for all of them.
template <int LPT, typename F>
__device__ __forceinline__ F token_sum(F v) {
    v += of_lane_xor<1>(v);
    v += of_lane_xor<2>(v);
    v += of_lane_xor<4>(v);
    v += of_lane_xor<8>(v);
    if constexpr (LPT == 32) v += of_lane_xor<16>(v);
    if constexpr (LPT == kWave) v = (of_lane(v, 0) + of_lane(v, 16)) + (of_lane(v, 32) + of_lane(v, 48));
    return v;
}
// The same for doubles, ordered as 64-bit integers in two halves: the largest high half, then the
// largest low half among the lanes that have it.
template <int LPT>
__device__ __forceinline__ double token_max(double v) {
    const int64_t b = __builtin_bit_cast(int64_t, v + 0.0);
    const int64_t o = b ^ ((b >> 63) & INT64_MAX);
    const int hi = token_max<LPT>((int)(o >> 32));
    const int lo = token_max<LPT>((int)(o >> 32) == hi ? (int)((uint32_t)o ^ 0x80000000u) : INT_MIN);
    const int64_t m = ((int64_t)hi << 32) | ((uint32_t)lo ^ 0x80000000u);
    return __builtin_bit_cast(double, m ^ ((m >> 63) & INT64_MAX));
}

// The token's lanes of a ballot, in its low bits.
template <int LPT>
__device__ __forceinline__ uint64_t token_bits(uint64_t ballot, int lane) {
    if constexpr (LPT == kWave) return ballot;
    return (ballot >> (lane & (kWave - LPT))) & ((1ull << LPT) - 1ull);
}

// A lane's part of its token.
template <int VPL>
struct Part {
    float logit[VPL];  // -inf: not to be chosen, whatever the bias
    float bias[VPL];   // -inf: not to be chosen
    int first;         // expert of element 0
};

// Which groups stay, as a bit each (a rating orders as `exact` or `rough` does, ties to the lower
// group), from lane g's rating of group g.  Returns in *close whether a group kept and one dropped
// are no further apart than one of their `slack`s.
template <int LPT, typename F>
__device__ __forceinline__ uint64_t keep_groups(F rating, int G, int kept, float slack, int lane, bool *close) {
    const int at = lane & (LPT - 1), base = lane & (kWave - LPT);
    auto rating_of = [&](int g) {
        if constexpr (sizeof(F) == 8)
            return LPT == kWave ? __builtin_bit_cast(double, readlane64(__builtin_bit_cast(uint64_t, rating), g))
                                : shfl_f64(rating, base + g);
        else
            return LPT == kWave ? readlanef(rating, g) : __shfl(rating, base + g);
    };
    int ahead = 0;  // groups rated above the lane's
    for (int g = 0; g < G; ++g) {
        const F o = rating_of(g);
        ahead += o > rating || (o == rating && g < at);
    }
    const bool stays = at < G && ahead < kept;
    const uint64_t bits = token_bits<LPT>(ballot64(stays), lane);
    if (close != nullptr) {
        bool near = false;
        for (int g = 0; g < G; ++g) {
            const float o = (float)rating_of(g);  // by all lanes, whether they need it or not
            near |= ((bits >> g) & 1ull) != (uint64_t)stays && !(fabsf(o - (float)rating) > slack);
        }
        // -inf (a group without experts to choose) is near nothing; a sum that overflows is near all
        near &= at < G && rating > -INFINITY;
        *close = token_bits<LPT>(ballot64(near), lane) != 0ull;
    }
    return bits;
}

// A slot's expert (-1: none) and what it was chosen by.
struct Chosen {
    int expert, key;
};

// Experts of a token that may have to be ordered anew: its slots, the one behind them and a few more.
constexpr int kCandidates = kMaxTopk + 8;

// The lane's choices in binary64 (-inf: not to be chosen).  choice (LDS): VPL values, kWave apart.  The
// logits go through LDS too, so that the exponentials are a loop: it is seldom run, and there are up to 32.
template <int LPT, int VPL>
__device__ __forceinline__ void exact_choices(const RouteParams &p, const Part<VPL> &t, double *choice) {
    const bool biased = p.a.bias != nullptr;
    int m = kNone;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int o = t.logit[i] > -INFINITY ? order_of(t.logit[i]) : kNone;
        m = o > m ? o : m;
        choice[i * kWave] = (double)t.logit[i];
    }
    m = token_max<LPT>(m);
    const double top = m == kNone ? 0.0 : (double)value_of(m);
    double sum = 0.0;
#pragma unroll 1
    for (int i = 0; i < VPL; ++i) {
        const double l = choice[i * kWave];
        double c = 0.0;
        if (l > -INFINITY) c = p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - top);
        choice[i * kWave] = c;
        sum += c;
    }
    sum = p.sigmoid ? 1.0 : token_sum<LPT>(sum);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const bool able = t.logit[i] > -INFINITY && t.bias[i] > -INFINITY;
        const double c = choice[i * kWave] / sum + (biased ? (double)t.bias[i] : 0.0);
        choice[i * kWave] = able ? c : -INFINITY;
    }
}

// Lane g: the rating of group g (-inf without experts), from the token's choices in LDS (those of the
// wave's lane l from choice[l], kWave apart).  group_lanes lanes share a group's experts.  *size: the
// sum of what the rating adds up, without signs.
template <int LPT, int VPL, typename V>
__device__ __forceinline__ V rate_groups(const RouteParams &p, const V *choice, int lane, float *size) {
    const int at = lane & (LPT - 1), base = lane & (kWave - LPT);
    const V none = -INFINITY;
    const int g = at / p.group_lanes;
    V a = none, b = none;
    if (g < p.G) {
        const int end = (g + 1) * p.group_size;
#pragma unroll 4
        for (int e = g * p.group_size + at % p.group_lanes; e < end; e += p.group_lanes) {
            const V v = choice[e % VPL * kWave + base + e / VPL];
            const V low = v < a ? v : a;
            a = v > a ? v : a;
            b = low > b ? low : b;
        }
    }
    auto join = [&](V oa, V ob) {
        const V low = a < oa ? a : oa;
        a = a > oa ? a : oa;
        b = b > ob ? b : ob;
        b = b > low ? b : low;
    };
    if (p.group_lanes > 1) join(of_lane_xor<1>(a), of_lane_xor<1>(b));
    if (p.group_lanes > 2) join(of_lane_xor<2>(a), of_lane_xor<2>(b));
    if (p.group_lanes > 4) join(of_lane_xor<4>(a), of_lane_xor<4>(b));
    if (p.group_lanes > 8) join(of_lane_xor<8>(a), of_lane_xor<8>(b));
    if (p.group_lanes > 16) join(of_lane_xor<16>(a), of_lane_xor<16>(b));
    const bool two = p.best == 2 && b > none;
    const V rating = two ? a + b : a;
    const int from = base + ((at * p.group_lanes) & (LPT - 1));
    V r;
    if constexpr (sizeof(V) == 8) {
        r = shfl_f64(rating, from);
    } else {
        r = __shfl(rating, from);
        *size = __shfl(two ? fabsf(a) + fabsf(b) : fabsf(a), from);
    }
    return at < p.G ? r : none;
}

// The num_topk largest choices in binary64, one after the other: where more experts are near each other
// than there are candidates.
template <int LPT, int VPL>
__device__ __forceinline__ void choose_exact(const RouteParams &p, int lane, double *choice, Chosen *chosen) {
    const int at = lane & (LPT - 1);
    const double none = -INFINITY;
#pragma unroll 1
    for (int j = 0; j < p.K; ++j) {
        double m = none;
        int e = 0;
#pragma unroll 1
        for (int i = 0; i < VPL; ++i) {
            const double v = choice[i * kWave];
            if (v > m) {
                m = v;
                e = i;
            }
        }
        const double best = token_max<LPT>(m);
        const uint64_t holders = token_bits<LPT>(ballot64(m == best && best > none), lane);
        if (holders == 0ull) {
            if (at == 0) chosen[j].expert = -1;
        } else if (at == __builtin_ctzll(holders)) {
            choice[e * kWave] = none;
            chosen[j].expert = at * VPL + e;
        }
    }
}

// The choice for the token whose logits start at element `row`.  chosen (LDS): its candidates, all
// without an expert before; the first num_topk are the choice.  value (LDS): a number for each.  exact
// (LDS): the wave's, VPL x kWave.
template <int LPT, int VPL, bool BF16>
__device__ __forceinline__ void choose(const RouteParams &p, const Part<VPL> &t, int64_t row, int lane,
                                       double (*exact)[kWave], Chosen *chosen, double *value) {
    const int at = lane & (LPT - 1);
    const bool biased = p.a.bias != nullptr;
    const bool by_logit = !biased && p.best == 1;  // what rates a group
    float slack = kSigmoidSlack;
    float choice[VPL];
    int key[VPL];
    if (biased || (p.G > 1 && !by_logit)) {
        float top = 0.0f, sum = 1.0f;
        if (!p.sigmoid) {
            int m = kNone;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int o = t.logit[i] > -INFINITY ? order_of(t.logit[i]) : kNone;
                m = o > m ? o : m;
            }
            m = token_max<LPT>(m);
            top = m == kNone ? 0.0f : value_of(m);
            sum = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            choice[i] = p.sigmoid ? 1.0f / (1.0f + expf(-t.logit[i])) : expf(t.logit[i] - top);  // -inf: 0
            sum += choice[i];
        }
        float scale = 1.0f;
        if (!p.sigmoid) {
            scale = 1.0f / token_sum<LPT>(sum);  // the largest score
            slack = kSoftmaxSlack * fminf(scale, 1.0f);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) choice[i] = __builtin_fmaf(choice[i], scale, biased ? t.bias[i] : 0.0f);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const bool able = t.logit[i] > -INFINITY && (!biased || t.bias[i] > -INFINITY);
        key[i] = able ? order_of(biased ? choice[i] : t.logit[i]) : kNone;
    }
    uint64_t keep = ~0ull;
    bool have_exact = false;
    if (p.G > 1) {
        float *rough = reinterpret_cast<float *>(&exact[0][0]);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            rough[i * kWave + lane] = key[i] == kNone ? -INFINITY : by_logit ? t.logit[i] : choice[i];
        wave_lds_order();
        float size;
        const float rating = rate_groups<LPT, VPL>(p, rough, lane, &size);
        wave_lds_order();
        bool close = false;
        // two choices and their sum's rounding on either side
        keep = keep_groups<LPT>(rating, p.G, p.kept, 2.0f * (slack + kSlack * size), lane, by_logit ? nullptr : &close);
        if (ballot64(close) != 0ull) {
            exact_choices<LPT, VPL>(p, t, &exact[0][lane]);
            have_exact = true;
            wave_lds_order();
            const double sure = rate_groups<LPT, VPL>(p, &exact[0][0], lane, nullptr);
            keep = keep_groups<LPT>(sure, p.G, p.kept, 0.0f, lane, nullptr);
        }
    }
    auto kept = [&](int e) {
        const int g = e / p.group_size;
        return g < p.G && ((keep >> g) & 1ull) != 0ull;
    };
    if (p.G > 1) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (!kept(t.first + i)) key[i] = kNone;
    }
    // a round: the largest key left, lowest expert first
    auto round = [&](int j) {
        int m = key[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) m = key[i] > m ? key[i] : m;
        const int best = token_max<LPT>(m);
        if (ballot64(best != kNone) == 0ull) return false;
        const uint64_t holders = token_bits<LPT>(ballot64(m == best && best != kNone), lane);
        const bool mine = holders != 0ull && at == __builtin_ctzll(holders | (1ull << 63));
        int e = 0;
        bool done = !mine;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool hit = !done && key[i] == best;
            key[i] = hit ? kNone : key[i];
            e = hit ? i : e;
            done |= hit;
        }
        if (mine) chosen[j] = {t.first + e, best};
        return true;
    };
    // num_topk rounds, and with a bias one more, to see how near it is
    const int rounds = p.K + (biased ? 1 : 0);
    for (int j = 0; j < rounds; ++j)
        if (!round(j)) break;
    wave_lds_order();
    if (!biased) return;

    auto near = [&](const Chosen &a, const Chosen &b) {
        const float v = value_of(a.key);
        return b.expert >= 0 && v - value_of(b.key) <= slack + kSlack * fabsf(v);
    };
    // Lane j: slots j and j + 1.  The same logit and bias are a tie in any precision; but those behind
    // the last slot may be followed by others that are not the same.
    bool close = false;
    for (int j = at; j < p.K; j += LPT) {
        const Chosen a = chosen[j], b = chosen[j + 1];
        if (near(a, b))
            close |= j + 1 == p.K || load_logit<BF16>(p.a.logits, row + a.expert) != load_logit<BF16>(p.a.logits, row + b.expert) ||
                     p.a.bias[a.expert] != p.a.bias[b.expert];
    }
    if (ballot64(close) == 0ull) return;
    int n = p.K + 1;
    bool open = near(chosen[n - 2], chosen[n - 1]);
    while (n < kCandidates && ballot64(open) != 0ull) {
        if (!round(n)) open = false;
        wave_lds_order();
        ++n;
        open = open && near(chosen[n - 2], chosen[n - 1]);
    }
    const bool overflow = ballot64(open) != 0ull;
    if ((overflow || !p.sigmoid) && !have_exact) {
        exact_choices<LPT, VPL>(p, t, &exact[0][lane]);
        have_exact = true;
    }
    wave_lds_order();
    if (overflow) {
#pragma unroll 1
        for (int i = 0; i < VPL; ++i)
            if (!kept(t.first + i)) exact[i][lane] = -INFINITY;
        choose_exact<LPT, VPL>(p, lane, &exact[0][lane], chosen);
        return;
    }
    constexpr int kMine = (kCandidates + LPT - 1) / LPT;  // a lane's candidates
    int place[kMine], expert[kMine];
    for (int j = at; j < n; j += LPT) {
        const int e = chosen[j].expert;
        double v = -INFINITY;
        if (e >= 0 && have_exact)
            v = exact[e % VPL][(lane & (kWave - LPT)) + e / VPL];
        else if (e >= 0)
            v = 1.0 / (1.0 + exp(-(double)load_logit<BF16>(p.a.logits, row + e))) + (double)p.a.bias[e];
        value[j] = v;
    }
    wave_lds_order();
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
        const int j = at + u * LPT;
        expert[u] = -1;
        place[u] = p.K;
        if (j >= n || chosen[j].expert < 0) continue;
        const double v = value[j];
        int ahead = 0;
        expert[u] = chosen[j].expert;
        for (int o = 0; o < n; ++o) {
            const int e = chosen[o].expert;
            ahead += e >= 0 && (value[o] > v || (value[o] == v && e < expert[u]));
        }
        place[u] = ahead;
    }
    wave_lds_order();
#pragma unroll
    for (int u = 0; u < kMine; ++u)
        if (place[u] < p.K) chosen[place[u]].expert = expert[u];
}

// One launch routes a token per LPT lanes.  128 tokens of 256 experts in 8 groups take 7.3 us on the card, a
// launch (about 3) included: latency, of loads, group ratings and a chain of cross-lane steps a slot.  16384
// tokens of 64 experts take 6 us, over the 0.6 that their bytes need, for the same reason.  Many tokens of many experts
// are bound by the selection, which looks through all of a lane's keys a round: 7747 tokens of 471 experts with a bias
// take 11.7 us for one slot and 17.5 for eight, 0.8 to 0.9 a slot.
template <int LPT, int VPL, bool BF16>
__global__ __launch_bounds__(kRouteWaves *kWave) void route_kernel(RouteParams p) {
    constexpr int kTokens = kWave / LPT;  // of a wave
    __shared__ Chosen s_chosen[kRouteWaves * kTokens][kCandidates];
    __shared__ double s_value[kRouteWaves * kTokens][kCandidates];
    __shared__ double s_exact[kRouteWaves][VPL][kWave];
    const int lane = threadIdx.x & (kWave - 1), at = lane & (LPT - 1);
    const int slot = threadIdx.x / LPT;  // the token's place in the block
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves * kTokens + slot;
    const bool here = t < p.T;
    const bool on = here && (p.a.token_mask == nullptr || p.a.token_mask[t] != 0);
    const int64_t row = t * p.a.stride;
    Part<VPL> part;
    part.first = at * VPL;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        part.logit[i] = -INFINITY;
        part.bias[i] = 0.0f;
    }
    if (on) load_logits<VPL, BF16>(p.a.logits, row + part.first, p.E - part.first, part.logit);
    if (p.a.bias != nullptr) load_values<VPL>(p.a.bias, part.first, p.E - part.first, part.bias);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        if (unusable(part.logit[i])) {
            bad = true;
            part.logit[i] = -INFINITY;
        }
        if (unusable(part.bias[i])) {
            bad |= on;
            part.bias[i] = -INFINITY;
        }
    }
    if (ballot64(bad) != 0ull && lane == 0) flag(p.a.dev_status, EP_DEV_BAD_LOGIT);

    for (int j = at; j < kCandidates; j += LPT) s_chosen[slot][j] = {-1, kNone};
    wave_lds_order();
    choose<LPT, VPL, BF16>(p, part, row, lane, s_exact[threadIdx.x / kWave], s_chosen[slot], s_value[slot]);
    wave_lds_order();

    // lane j: slot j (num_topk <= LPT, which the launcher sees to).  In 64 bits: there are few of them
    const int chosen = at < p.K ? s_chosen[slot][at].expert : -1;
    double s = 0.0;
    if (chosen >= 0) {
        // with no bias the logit is what it was chosen by
        const double l = p.a.bias == nullptr ? value_of(s_chosen[slot][at].key) : load_logit<BF16>(p.a.logits, row + chosen);
        s = p.sigmoid ? 1.0 / (1.0 + exp(-l)) : l;
    }
    if (!p.sigmoid) {
        // relative to the largest logit of the row, or of the chosen ones where only their ratios count
        double ref = chosen >= 0 ? s : -INFINITY, sum = 1.0;
        if (p.renorm) {
            ref = token_max<LPT>(ref);
        } else {
            int m = kNone;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int o = part.logit[i] > -INFINITY ? order_of(part.logit[i]) : kNone;
                m = o > m ? o : m;
            }
            m = token_max<LPT>(m);
            const float top = m == kNone ? 0.0f : value_of(m);
            // in f32, off by under 56 * 2^-24; in 64 bits 16384 tokens of 64 experts take 6.8 us for 6.4, of 256 16.4 for 14.4
            float all = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) all += expf(part.logit[i] - top);
            ref = (double)top;
            sum = (double)token_sum<LPT>(all);
        }
        s = chosen >= 0 ? exp(s - ref) / sum : 0.0;
    }
    double w = s * (double)p.scale;
    if (p.renorm) {
        const double all = token_sum<LPT>(s);
        w = all > 0.0 ? w / all : 0.0;
    }
    if (here && at < p.K) {
        p.a.topk_idx[t * p.K + at] = chosen;
        p.a.topk_w[t * p.K + at] = (float)w;
    }
}

// VPL experts a lane at a time, all of a token's at once where they fit.  4096 tokens of 256 experts take 5.7 us on
// the card (sigmoid, renormalised; 8.8 MB, 1.7 us of bytes), 16384 tokens of 64 in bf16 6.7 us (softmax, not
// renormalised): a launch and the latency of one wave's loads, sums over its slots and stores.
template <int LPT, int VPL, bool BF16>
__global__ __launch_bounds__(kRouteWaves *kWave) void route_backward_kernel(RouteBackwardParams p) {
    constexpr int kTokens = kWave / LPT, kSpan = LPT * VPL;
    const int lane = threadIdx.x & (kWave - 1), at = lane & (LPT - 1), base = lane & (kWave - LPT);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves * kTokens + threadIdx.x / LPT;
    const bool here = t < p.T;
    const int64_t row = t * p.a.stride;
    // lane j: slot j's expert (num_topk <= LPT, which the launcher sees to)
    int id = -1;
    bool bad_id = false;
    if (here && at < p.K) {
        const int64_t e = p.a.topk_idx[t * p.K + at];
        bad_id = e < -1 || e >= p.E;
        if (e >= 0 && e < p.E) id = (int)e;
    }
    if (ballot64(bad_id) != 0ull && lane == 0) flag(p.a.dev_status, EP_DEV_BAD_TOPK_IDX);
    // a token without slots has a gradient of zeros, whatever its logits: they are not read
    const bool on = token_bits<LPT>(ballot64(id >= 0), lane) != 0ull;
    float logit[VPL];
    bool bad = false;
    auto load = [&](int from) {  // -inf where there is no usable logit
#pragma unroll
        for (int i = 0; i < VPL; ++i) logit[i] = -INFINITY;
        const int e = from + at * VPL;
        if (on) load_logits<VPL, BF16>(p.a.logits, row + e, p.E - e, logit);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            if (unusable(logit[i])) {
                bad = true;
                logit[i] = -INFINITY;
            }
        }
    };
    // a softmax that is not renormalised: the largest logit and the sum relative to it
    const bool whole_row = !p.sigmoid && !p.renorm;
    float top = 0.0f, sum = 1.0f;
    load(0);
    if (whole_row) {
        int m = kNone;
        for (int from = 0; from < p.E; from += kSpan) {
            if (from > 0) load(from);
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                const int o = logit[i] > -INFINITY ? order_of(logit[i]) : kNone;
                m = o > m ? o : m;
            }
        }
        m = token_max<LPT>(m);
        top = m == kNone ? 0.0f : value_of(m);
        sum = 0.0f;
        for (int from = 0; from < p.E; from += kSpan) {
            if (p.E > kSpan) load(from);
#pragma unroll
            for (int i = 0; i < VPL; ++i) sum += expf(logit[i] - top);
        }
        sum = token_sum<LPT>(sum);
    }

    // Lane j: what slot j adds to its expert's logit, whole in 64 bits and rounded once.  The gradient of a score
    // is as large as the score is small, and the sums over the slots cancel: neither part alone fits 32 bits.
    double s = 0.0, rest = 1.0, g = 0.0;  // the score, 1 - score (a sigmoid's), the weight's gradient
    float l = -INFINITY;
    if (id >= 0) {
        l = load_logit<BF16>(p.a.logits, row + id);
        if (unusable(l)) l = -INFINITY;
        g = p.a.grad_w[t * p.K + at];
    }
    double ref = (double)top;
    if (!p.sigmoid && p.renorm) {  // only the ratios of the chosen ones' scores count
        const int m = token_max<LPT>(l > -INFINITY ? order_of(l) : kNone);
        ref = m == kNone ? 0.0 : (double)value_of(m);
    }
    if (l > -INFINITY) {
        if (p.sigmoid) {
            s = 1.0 / (1.0 + exp(-(double)l));
            rest = 1.0 / (1.0 + exp((double)l));  // does not cancel where s is near 1
        } else {
            s = exp((double)l - ref) / (double)sum;
        }
    }
    const double scale = (double)p.scale;
    double part, mean = 0.0;  // mean: sum over the slots of ds s, which every logit of a softmax gets its score's share of
    if (p.renorm) {
        const double all = token_sum<LPT>(s), r = all > 0.0 ? s / all : 0.0;
        part = scale * (g - token_sum<LPT>(g * r)) * r;  // and these have a mean of 0
    } else {
        part = scale * g * s;
        if (whole_row) {
            mean = token_sum<LPT>(part);
            part -= mean * s;
        }
    }
    const float slot = (float)(part * rest);
    const float share = (float)mean;

    for (int from = 0; from < p.E; from += kSpan) {
        if (p.E > kSpan) load(from);
        const int e0 = from + at * VPL;
        float d[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) d[i] = 0.0f;
        uint32_t named = 0, again = 0;  // elements in a slot, and in one more
        for (int j = 0; j < p.K; ++j) {
            const int e = (LPT == kWave ? readlane32(id, j) : __shfl(id, base + j)) - e0;
            const float v = LPT == kWave ? readlanef(slot, j) : __shfl(slot, base + j);
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (e == i) d[i] += v;
            const uint32_t bit = (uint32_t)e < VPL ? 1u << e : 0u;
            again |= named & bit;
            named |= bit;
        }
        if (whole_row) {
            // the mean's share: experts without a slot lose it here, of the others each slot has lost it
            float lost[VPL];
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                lost[i] = expf(logit[i] - top) / sum * share;
                if ((named >> i & 1u) == 0u) d[i] = -lost[i];
            }
            if (ballot64(again != 0u) != 0ull) {  // and those in several slots get it back but for once
                named = 0;
                for (int j = 0; j < p.K; ++j) {
                    const int e = __shfl(id, base + j) - e0;
#pragma unroll
                    for (int i = 0; i < VPL; ++i) {
                        if (e != i) continue;
                        if ((named >> i & 1u) != 0u) d[i] += lost[i];
                        named |= 1u << i;
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (logit[i] == -INFINITY) d[i] = 0.0f;
        if (!here) continue;
        const int64_t out = t * p.a.grad_stride + e0;
        store_logits<VPL, BF16>(p.a.grad_logits, out, p.E - e0, d);
    }
    if (ballot64(bad) != 0ull && lane == 0) flag(p.a.dev_status, EP_DEV_BAD_LOGIT);
}

template <int LPT, int VPL, bool BF16>
hipError_t start(RouteParams p, hipStream_t stream) {
    constexpr int kTokens = kRouteWaves * kWave / LPT;
    p.group_lanes = 1;
    while (2 * p.group_lanes * p.G <= LPT) p.group_lanes *= 2;
    return start_kernel(route_kernel<LPT, VPL, BF16>, (p.T + kTokens - 1) / kTokens, kRouteWaves * kWave, stream, p);
}
template <int LPT, int VPL, bool BF16>
hipError_t start(RouteBackwardParams p, hipStream_t stream) {
    constexpr int kTokens = kRouteWaves * kWave / LPT;
    return start_kernel(route_backward_kernel<LPT, VPL, BF16>, (p.T + kTokens - 1) / kTokens, kRouteWaves * kWave, stream, p);
}

template <bool BF16>
hipError_t start_route(const RouteParams &p, hipStream_t stream) {
    if (p.T >= kManyTokens) {
        const bool narrow = p.K <= 16 && p.G <= 16;  // slots and groups have a lane each
        if (narrow && p.E <= 64) return start<16, 4, BF16>(p, stream);
        if (narrow && p.E <= 128) return start<16, 8, BF16>(p, stream);
        if (p.G <= 32 && p.E > 128 && p.E <= 256) return start<32, 8, BF16>(p, stream);
    }
    if (p.E <= 64) return start<64, 1, BF16>(p, stream);
    if (p.E <= 128) return start<64, 2, BF16>(p, stream);
    if (p.E <= 256) return start<64, 4, BF16>(p, stream);
    if (p.E <= 512) return start<64, 8, BF16>(p, stream);
    if (p.E <= 1024) return start<64, 16, BF16>(p, stream);
    return start<64, 32, BF16>(p, stream);
}

template <bool BF16>
hipError_t start_backward(const RouteBackwardParams &p, hipStream_t stream) {
    if (p.T >= kManyTokens) {
        if (p.K <= 16 && p.E <= 64) return start<16, 4, BF16>(p, stream);
        if (p.K <= 16 && p.E <= 128) return start<16, 8, BF16>(p, stream);
        if (p.E > 128 && p.E <= 256) return start<32, 8, BF16>(p, stream);
    }
    if (p.E <= 64) return start<64, 1, BF16>(p, stream);
    if (p.E <= 128) return start<64, 2, BF16>(p, stream);
    return start<64, 4, BF16>(p, stream);
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
    return a.bf16 ? start_route<true>(p, stream) : start_route<false>(p, stream);
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
    return a.bf16 ? start_backward<true>(p, stream) : start_backward<false>(p, stream);
}

}  // namespace ep
