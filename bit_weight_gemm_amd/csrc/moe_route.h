// A mixture's router, in the registers of one wave: what moe_route.hip's kernel and a whole layer's share (gfx950).
#pragma once

#include <type_traits>

#include "q4.h"

namespace tq2 {

__device__ __forceinline__ float wave_sum(float v) {
    v = row16_sum(v);
    float a = v, b = v;
    swap16(a, b);
    v = a + b;
    a = v, b = v;
    swap32(a, b);
    return a + b;
}

template <int CTRL>
__device__ __forceinline__ int dppi(int v) {
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, false);
}
// v of the lane in the other half of each pair of 16-lane rows, or of the wave: the
// swap leaves one operand with the lower half's values in both, the other the upper's.
__device__ __forceinline__ int2 both16(int v) {
    const auto r = __builtin_amdgcn_permlane16_swap((unsigned)v, (unsigned)v, false, false);
    return int2{(int)r[0], (int)r[1]};
}
__device__ __forceinline__ int2 both32(int v) {
    const auto r = __builtin_amdgcn_permlane32_swap((unsigned)v, (unsigned)v, false, false);
    return int2{(int)r[0], (int)r[1]};
}
template <typename I>
__device__ __forceinline__ I imax(I a, I b) {
    return a > b ? a : b;
}
template <typename I>
__device__ __forceinline__ I imin(I a, I b) {
    return a < b ? a : b;
}

// Maximum over the wave, as a scalar: over each row of 16 lanes in DPP, then of the four rows.
template <typename I>
__device__ __forceinline__ I wave_imax(I v) {
    v = imax(v, (I)dppi<0xB1>((int)v));
    v = imax(v, (I)dppi<0x4E>((int)v));
    v = imax(v, (I)dppi<0x141>((int)v));
    v = imax(v, (I)dppi<0x140>((int)v));
    const I a = (I)__builtin_amdgcn_readlane((int)v, 0), b = (I)__builtin_amdgcn_readlane((int)v, 16);
    const I c = (I)__builtin_amdgcn_readlane((int)v, 32), d = (I)__builtin_amdgcn_readlane((int)v, 48);
    return imax(imax(a, b), imax(c, d));
}

__device__ __forceinline__ double dpp_sum16(double v) {
    auto add = [&](auto f) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        v += __builtin_bit_cast(double, (uint64_t)(uint32_t)f((int)(b >> 32)) << 32 | (uint32_t)f((int)b));
    };
    add(dppi<0xB1>), add(dppi<0x4E>), add(dppi<0x141>), add(dppi<0x140>);  // exchanges: every lane's sum has the same bits
    return v;
}

__device__ __forceinline__ double wave_sum(double v) {
    v = dpp_sum16(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

__device__ __forceinline__ float uniform(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

constexpr float kNone = -__builtin_inff();
constexpr int kGone = -0x7fffffff - 1;  // below every key

// Integers that order as the floats do (-0 as 0, NaN above all).
__device__ __forceinline__ int order_of(float v) {
    const int b = __builtin_bit_cast(int, v + 0.0f);
    return v != v ? 0x7fffffff : b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int o) { return __builtin_bit_cast(float, o ^ ((o >> 31) & 0x7fffffff)); }
__device__ __forceinline__ int64_t order_of(double v) {
    const int64_t b = __builtin_bit_cast(int64_t, v + 0.0);
    return v != v ? 0x7fffffffffffffff : b ^ ((b >> 63) & 0x7fffffffffffffff);
}
__device__ __forceinline__ double value_of(int64_t o) {
    return __builtin_bit_cast(double, o ^ ((o >> 63) & 0x7fffffffffffffff));
}
constexpr int kNoneOrder = (int)0x807fffff;  // order_of(-inf)
constexpr int64_t kNoneOrder64 = (int64_t)0x800fffffffffffff, kGone64 = -0x7fffffffffffffff - 1;

// The largest float of the wave (NaN is passed over), as a scalar.
__device__ __forceinline__ float wave_max(float v) { return value_of(wave_imax(v != v ? kNoneOrder : order_of(v))); }

// Maximum of 64-bit orders over the wave: the upper halves, then the lower ones of those.
__device__ __forceinline__ int64_t wave_imax(int64_t v) {
    const int hi = (int)(v >> 32), m = wave_imax(hi);
    const uint32_t lo = wave_imax(hi == m ? (uint32_t)v : 0u);
    return (int64_t)((uint64_t)(uint32_t)m << 32 | lo);
}

template <bool SIGMOID>
__device__ __forceinline__ double score64(float l, float most, double total) {
    if (l == kNone) return 0.0;
    return SIGMOID ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)most) / total;
}

// exp of v to about two steps of f32 (v limited to +-88, where it is next to 0 or 2^127):
// the product with log2(e) in two parts around the hardware's exp2.  NaN stays (the limits would drop it).
__device__ __forceinline__ float exp_of(float x) {
    const float v = __builtin_amdgcn_fmed3f(x, -88.0f, 88.0f);
    const float t = v * 1.44269504f;
    const float rest = __builtin_fmaf(v, 1.92596299e-8f, __builtin_fmaf(v, 1.44269504f, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return x != x ? x : __builtin_fmaf(e, rest * 0.69314718f, e);
}

// (a, b) and (c, d), each the best two of a set, to the best two of both.
template <typename I>
__device__ __forceinline__ void merge2(I &a, I &b, I c, I d) {
    b = imax(imin(a, c), imax(b, d));
    a = imax(a, c);
}

// The best two of each group of 2^log_lanes lanes, in all its lanes.
__device__ __forceinline__ void best_two(int &a, int &b, int log_lanes) {
    if (log_lanes > 0) merge2(a, b, dppi<0xB1>(a), dppi<0xB1>(b));    // lane ^ 1
    if (log_lanes > 1) merge2(a, b, dppi<0x4E>(a), dppi<0x4E>(b));    // lane ^ 2
    if (log_lanes > 2) merge2(a, b, dppi<0x141>(a), dppi<0x141>(b));  // mirrored in eight lanes
    if (log_lanes > 3) merge2(a, b, dppi<0x140>(a), dppi<0x140>(b));  // mirrored in sixteen
    if (log_lanes > 4) {
        const int2 p = both16(a), q = both16(b);
        a = p.x, b = q.x;
        merge2(a, b, p.y, q.y);
    }
    if (log_lanes > 5) {
        const int2 p = both32(a), q = both32(b);
        a = p.x, b = q.x;
        merge2(a, b, p.y, q.y);
    }
}
__device__ __forceinline__ void best_two(int64_t &a, int64_t &b, int log_lanes) {
    for (int o = 0; o < log_lanes; ++o) merge2(a, b, (int64_t)__shfl_xor(a, 1 << o), (int64_t)__shfl_xor(b, 1 << o));
}

// Where a lane's experts lie: expert(c) = first + c * lanes for c < own.
struct Place {
    int lanes, group, first, own;
};

// A lane's keys in falling order, equal ones by expert (V <= 4: exchanges of neighbours; more: none,
// take_best looks for the largest).  from[i]: which of the lane's experts key[i] is.
template <int V, typename I>
__device__ __forceinline__ void sort_keys(I (&key)[V], int (&from)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) from[i] = i;
    if constexpr (V > 1 && V <= 4) {
#pragma unroll
        for (int pass = 0; pass + 1 < V; ++pass)
#pragma unroll
            for (int i = 0; i + 1 < V - pass; ++i)
                if (key[i + 1] > key[i]) {
                    const I k = key[i];
                    key[i] = key[i + 1], key[i + 1] = k;
                    const int f = from[i];
                    from[i] = from[i + 1], from[i + 1] = f;
                }
    }
}

// One pass over the keys (sort_keys'): the largest, with the lowest expert among equal
// ones, goes.  Returns the expert (-1: none is left) and its key.
template <int V, typename I>
__device__ __forceinline__ int take_best(I (&key)[V], int (&from)[V], const Place &at, int lane, I none, I gone, I &best) {
    I top = key[0];
    int c = from[0], pos = 0;
    if constexpr (V > 4) {
#pragma unroll
        for (int i = 1; i < V; ++i)
            if (key[i] > top) top = key[i], c = i, pos = i;
    }
    best = wave_imax(top);
    if (best <= none) return -1;
    const int mine = at.first + c * at.lanes;
    uint64_t who = __ballot(top == best);
    if (who & (who - 1)) {  // several lanes: the lowest expert
        const int low = -wave_imax(top == best ? -mine : kGone);
        who = __ballot(top == best && mine == low);
    }
    const int w = __builtin_ctzll(who);
    if constexpr (V > 4) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane == w && pos == i) key[i] = gone;
    } else if (lane == w) {
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1], from[i] = from[i + 1];
        key[V - 1] = gone;
    }
    return __builtin_amdgcn_readlane(mine, w);
}

// Whether this lane's group is one of the `keep` with the largest keys (own: the group's key).
template <typename I>
__device__ __forceinline__ bool stays(const RouteArgs &p, I own, const Place &at, int log_lanes) {
    int place = 0;
    for (int q = 0; q < p.groups; ++q) {
        I v;
        if constexpr (sizeof(I) == 8) {
            const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)own, q << log_lanes);
            const uint32_t hi = __builtin_amdgcn_readlane((int)(own >> 32), q << log_lanes);
            v = (I)((uint64_t)hi << 32 | lo);
        } else {
            v = __builtin_amdgcn_readlane(own, q << log_lanes);
        }
        if (v > own || (v == own && q < at.group)) ++place;
    }
    return at.group < p.groups && place < p.keep;
}

// Slots of one token in f64; lane j < k gets slot j's expert.
template <int V, bool SIGMOID>
__device__ inline int route_exact(const RouteArgs &p, const float (&l)[V], float most, const Place &at, int log_lanes, int lane) {
    int64_t key[V];
    double total = 1.0;
    if constexpr (!SIGMOID) {
        total = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) total += l[i] == kNone ? 0.0 : exp((double)l[i] - (double)most);
        total = wave_sum(total);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        double v = score64<SIGMOID>(l[i], most, total);
        if (p.bias && i < at.own) v += (double)p.bias[at.first + i * at.lanes];
        key[i] = i < at.own && l[i] != kNone ? order_of(v) : kNoneOrder64;
    }
    if (p.groups > 1) {
        int64_t a = kNoneOrder64, b = kNoneOrder64;
#pragma unroll
        for (int i = 0; i < V; ++i) merge2(a, b, key[i], kNoneOrder64);
        best_two(a, b, log_lanes);
        if (p.group_top > 1 && b > kNoneOrder64) a = order_of(value_of(a) + value_of(b));
        if (!stays(p, a, at, log_lanes)) {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = kNoneOrder64;
        }
    }
    int mine = -1, from[V];
    sort_keys<V>(key, from);
    for (int j = 0; j < p.k; ++j) {
        int64_t best;
        const int e = take_best<V, int64_t>(key, from, at, lane, kNoneOrder64, kGone64, best);
        if (e < 0) break;
        if (lane == j) mine = e;
    }
    return mine;
}

// Lanes of a group, as a power of two: the most that 64 have for each.
inline int route_log_lanes(int groups) {
    int log_lanes = 6;
    while ((groups << log_lanes) > 64) --log_lanes;
    return log_lanes;
}
// Experts of a lane.
inline int route_own(int E, int groups) {
    const int log_lanes = route_log_lanes(groups);
    return (E / groups + (1 << log_lanes) - 1) >> log_lanes;
}

__device__ __forceinline__ Place route_place(const RouteArgs &p, int log_lanes, int lane) {
    Place at;
    at.lanes = 1 << log_lanes, at.group = lane >> log_lanes;
    const int i0 = lane & (at.lanes - 1);
    at.first = at.group * p.n + i0;
    at.own = at.group < p.groups && i0 < p.n ? (p.n - i0 + at.lanes - 1) >> log_lanes : 0;
    return at;
}

// One token's experts, by one wave: lane j < k gets slot j's (-1: none).  l: the lane's logits, key: their biases (used up).
// V: experts per lane.  KEYS: keys are sums of scores, else the logits.  most and total: what the weights need of a softmax
// (total only if `weigh`).
template <int V, bool KEYS, bool SIGMOID>
__device__ __forceinline__ int route_choose(const RouteArgs &p, float (&l)[V], float (&key)[V], const Place &at, int log_lanes,
                                            int lane, bool weigh, float &most, float &total) {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = i < at.own ? l[i] : kNone;
    int order[V];  // of the keys: decides among experts
    most = kNone, total = 1.0f;
    if constexpr (!SIGMOID) {
        float m = l[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
        most = wave_max(m);
    }
    float error = 0.0f;  // bound on a key's error
    if constexpr (KEYS || !SIGMOID) {
        float score[V];
        if (!SIGMOID && (KEYS || weigh)) {
            float sum[V];
#pragma unroll
            for (int i = 0; i < V; ++i) sum[i] = score[i] = l[i] == kNone ? 0.0f : KEYS ? exp_of(l[i] - most) : expf(l[i] - most);
#pragma unroll
            for (int o = 1; o < V; o <<= 1)  // pairs of pairs: log2(V) roundings, not V - 1
#pragma unroll
                for (int i = 0; i < V; i += 2 * o) sum[i] += sum[i + o];
            // one lane's sum for all: the lanes' orders of addition differ
            total = uniform(wave_sum(sum[0]), 0);
        }
        if constexpr (KEYS) {
            float mag = 0.0f;
            const float inv = 1.0f / total;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float sc = SIGMOID ? __builtin_amdgcn_rcpf(1.0f + exp_of(-l[i])) : score[i] * inv;
                key[i] += sc;
                const float m = sc + __builtin_fabsf(key[i]);
                if (l[i] != kNone && m < __builtin_inff()) mag = fmaxf(mag, m);
            }
            // In steps of 2^-24 of the score, and one of the key for its sum with the bias.  exp_of: 3.2.
            // Sigmoid: the sum with 1 one more, the reciprocal two: 8 with that of a group's two keys.
            // Softmax: the rounded argument 0.4 of the largest score, and 5 of the total (the mean of
            // x e^-x over 1024 terms at most); the total's log2(V) and 6 additions; its terms 3.2; quotient
            // and product two: log2(V) + 22 likewise.  Scores below f32's normal range are flushed or held at
            // e^-88: at most 2^-126 each.
            error = (SIGMOID ? 8 : 22 + __builtin_ctz(V)) * 0x1p-24f * wave_max(mag) + 0x1p-125f;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        order[i] = order_of(l[i]);
        if constexpr (KEYS) {
            order[i] = order[i] == kNoneOrder ? kNoneOrder : order_of(key[i]);
        }
    }
    bool close = false;  // some decision within the keys' error
    if (p.groups > 1) {
        int a = kNoneOrder, b = kNoneOrder;
#pragma unroll
        for (int i = 0; i < V; ++i) merge2(a, b, order[i], kNoneOrder);
        best_two(a, b, log_lanes);
        if (p.group_top > 1 && b > kNoneOrder) a = order_of(value_of(a) + value_of(b));
        const bool in = stays(p, a, at, log_lanes);
        if (KEYS && p.keep < p.groups) {
            const float low = value_of(-wave_imax(in ? -a : kGone)), high = value_of(wave_imax(!in ? a : kGone));
            close = low - high <= 4.0f * error;
        }
        if (!in) {
#pragma unroll
            for (int i = 0; i < V; ++i) order[i] = kNoneOrder;
        }
    }

    int mine = -1, from[V];
    sort_keys<V>(order, from);
    const int passes = KEYS ? p.k + 1 : p.k;  // one more key, to see how near it comes
    float before = 0.0f;
    for (int j = 0; j < passes; ++j) {
        int best;
        const int e = take_best<V, int>(order, from, at, lane, kNoneOrder, kGone, best);
        if (e < 0) break;
        if constexpr (KEYS) {
            if (j && before - value_of(best) <= 2.0f * error) close = true;
            before = value_of(best);
        }
        if (lane == j && j < p.k) mine = e;
    }
    if constexpr (KEYS) {
        if (close) mine = route_exact<V, SIGMOID>(p, l, most, at, log_lanes, lane);  // wave-uniform
    }
    return mine;
}

// Lane j's weight, from its expert's logit; the chosen scores in f64, one per lane.
template <bool SIGMOID>
__device__ __forceinline__ float route_weight(const RouteArgs &p, int mine, float chosen, float most, float total) {
    double w = mine < 0 ? 0.0 : score64<SIGMOID>(chosen, most, (double)total);
    if (p.renorm) {
        const double sum = p.k <= 16 ? dpp_sum16(w) : wave_sum(w);
        if (sum != 0.0) w /= sum;
    }
    return (float)w;
}

// One token's experts and weights from its f32 logits; `weigh`: the weights too.
struct Slot {
    int expert;
    float weight;
};
template <int V>
__device__ __forceinline__ Slot route_token(const RouteArgs &p, const float *logits, int log_lanes, int lane, bool weigh) {
    const Place at = route_place(p, log_lanes, lane);
    const bool keys = p.bias || (p.groups > 1 && p.group_top > 1);
    float l[V], key[V], most, total;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i < at.own ? at.first + i * at.lanes : 0;
        l[i] = logits[e];
        key[i] = p.bias ? p.bias[e] : 0.0f;
    }
    Slot s{};
    auto choose = [&](auto with_keys, auto sigmoid) {
        constexpr bool KEYS = decltype(with_keys)::value, SIGMOID = decltype(sigmoid)::value;
        s.expert = route_choose<V, KEYS, SIGMOID>(p, l, key, at, log_lanes, lane, weigh, most, total);
        if (weigh) s.weight = route_weight<SIGMOID>(p, s.expert, logits[s.expert < 0 ? 0 : s.expert], most, total);
    };
    using std::false_type;
    using std::true_type;
    if (keys && p.sigmoid) choose(true_type{}, true_type{});
    else if (keys) choose(true_type{}, false_type{});
    else if (p.sigmoid) choose(false_type{}, true_type{});
    else choose(false_type{}, false_type{});
    return s;
}

}  // namespace tq2
