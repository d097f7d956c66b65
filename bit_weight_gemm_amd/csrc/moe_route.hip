// A mixture's router: scores, groups, the k chosen experts and their weights, and
// the gradient of the weights with respect to the logits.
//
// Score p_e = softmax(l)_e or sigmoid(l_e); an expert's key is its logit (no bias and
// no sum of several keys per group: softmax and sigmoid are monotonic), else p_e +
// bias_e in f64.  A group's key is the sum of its group_top best keys; the `keep` best groups
// stay.  Among what is left the k largest keys are chosen, the first at slot 0; equal
// keys go to the lower index.  weights[j] = p of slot j's expert, divided by the sum
// over the slots if renorm.
//
// A logit of -inf masks its expert (so does a bias of -inf, or a dropped group):
// it is never chosen, and slots that find no expert get idx -1 and weight 0, which
// the experts' products skip.  A NaN key ranks first, so that it shows.
//
// Keys that are sums of scores decide whole numbers in near ties: over 16384 tokens of
// 256 experts f32 scores swap a pair every few calls, so such keys count in f64.  They
// are formed in f32 first, with a bound on their error; a token whose decisions (the
// order of its first k + 1 keys, and which groups stay) all have more than that
// between them is done, the others, a few in a thousand, are done again in f64.  (The
// logits' own order would not do inside groups either: different logits may have equal scores.)
//
// One wave per token.  A group has 2^log_lanes lanes, each with every 2^log_lanes-th of
// its experts, so a group's best keys are found in its own lanes.  Keys are compared as
// integers that order like them: a wave maximum is then six DPP instructions, and a pass
// for one slot about thirty.
//
// Bound by instruction issue: 16384 tokens x 256 experts, 8 groups of which 4 stay, bias, 8 chosen:
// 24-26 us of kernel (0.7 TB/s), some 600 vector instructions a token; one token 4.4-4.8 us, of which an
// empty launch is two.  The gradient reads and writes its rows once: 8192 x 128 f32 4.6-5.6 us (2 TB/s).
#include "q4.h"

namespace tq2 {

namespace {

constexpr int kWaves = 4;  // tokens per workgroup

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
__device__ int route_exact(const RouteArgs &p, const float (&l)[V], float most, const Place &at, int log_lanes, int lane) {
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

// V: experts per lane.  KEYS: keys are sums of scores, else the logits.
template <int DT, int V, bool KEYS, bool SIGMOID>
__global__ __launch_bounds__(kWaves * 64) void route_kernel(RouteArgs p, int log_lanes) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= p.T) return;
    const int n = p.n;
    Place at;
    at.lanes = 1 << log_lanes, at.group = lane >> log_lanes;
    const int i0 = lane & (at.lanes - 1);
    at.first = at.group * n + i0;
    at.own = at.group < p.groups && i0 < n ? (n - i0 + at.lanes - 1) >> log_lanes : 0;

    float l[V], key[V];
    int order[V];  // of the keys: decides among experts
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i < at.own ? at.first + i * at.lanes : 0;
        l[i] = load_as_float<DT>(p.logits, t * p.E + e);
        key[i] = KEYS && p.bias ? p.bias[e] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = i < at.own ? l[i] : kNone;
    float most = kNone, total = 1.0f;
    if constexpr (!SIGMOID) {
        float m = l[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
        most = wave_max(m);
    }
    float error = 0.0f;  // bound on a key's error
    if constexpr (KEYS || !SIGMOID) {
        float score[V];
        if constexpr (!SIGMOID) {
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
    // the chosen scores in f64, one per lane
    const float chosen = load_as_float<DT>(p.logits, t * p.E + (mine < 0 ? 0 : mine));
    double w = mine < 0 ? 0.0 : score64<SIGMOID>(chosen, most, (double)total);
    if (p.renorm) {
        const double sum = p.k <= 16 ? dpp_sum16(w) : wave_sum(w);
        if (sum != 0.0) w /= sum;
    }
    if (lane < p.k) {
        p.idx[t * p.k + lane] = mine;
        p.weights[t * p.k + lane] = (float)w;
    }
}

// dlogits of one token from its chosen experts' d(weights) dw_j, with p the scores.  Without renorm
// dp = dw scattered to the experts, then through softmax dl = p (dp - sum dp p), or sigmoid dl = dp p (1 - p).
// With renorm w_j = p_j / sum p over the slots, and the scores themselves cancel: dw/dl is softmax's among the
// chosen, w_j (dw_j - sum w_i dw_i), for sigmoid times 1 - p_j, and 0 for the others.  w is formed from exponents
// relative to the largest chosen logit, so that scores below f32's range have their gradient.
template <int DT, int V, bool SIGMOID>
__global__ __launch_bounds__(kWaves * 64) void route_backward_kernel(const void *logits, const int32_t *idx, const float *dw,
                                                                     void *dlogits, int64_t T, int E, int k, int renorm) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= T) return;
    int e = -1;
    float dc = 0.0f, c = kNone;  // of the lane's slot: d(weight), then what goes to its expert; its logit
    if (lane < k) {
        e = idx[t * k + lane];
        if (e < 0 || e >= E) e = -1;
        else {
            dc = dw[t * k + lane];
            c = load_as_float<DT>(logits, t * E + e);
        }
    }
    float l[V], pr[V];  // pr: softmax's scores, or sigmoid's factors
    float most = kNone, total = 1.0f, inv = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int x = lane + 64 * i;
        l[i] = x < E ? load_as_float<DT>(logits, t * E + x) : kNone;
        most = fmaxf(most, l[i]);
    }
    if constexpr (SIGMOID) {
#pragma unroll
        for (int i = 0; i < V; ++i) {  // p (1 - p), or with renorm 1 - p: from e^-|l|, where 1 - p would cancel
            const float a = expf(-__builtin_fabsf(l[i])), b = 1.0f / (1.0f + a);
            pr[i] = renorm ? (l[i] > 0.0f ? a * b : b) : a * b * b;
        }
    } else {
        most = wave_max(most);
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) total += pr[i] = l[i] == kNone ? 0.0f : expf(l[i] - most);
        total = wave_sum(total);
        inv = total == 0.0f ? 0.0f : 1.0f / total;  // 0: every logit is -inf
#pragma unroll
        for (int i = 0; i < V; ++i) pr[i] *= inv;
    }
    float dot = 0.0f;
    if (renorm) {
        const float top = wave_max(c), from = SIGMOID ? fminf(top, 0.0f) : top;
        float w = c == kNone ? 0.0f : SIGMOID && c >= 0.0f ? 1.0f : expf(c - from);
        if constexpr (SIGMOID) w /= 1.0f + expf(-__builtin_fabsf(c));
        bool none = top == kNone;
        if (!none && (SIGMOID ? top : top - most) < -700.0f)  // the forward's weights are 0 where the f64 scores are
            none = !__any(e >= 0 && score64<SIGMOID>(c, most, (double)total) > 0.0);
        const float sum = wave_sum(w);
        w = none || e < 0 ? 0.0f : w / sum;
        dc = w * (dc - wave_sum(w * dc));
    } else if constexpr (!SIGMOID) {
        dot = wave_sum(c == kNone ? 0.0f : dc * expf(c - most) * inv);
    }
    float dp[V];
#pragma unroll
    for (int i = 0; i < V; ++i) dp[i] = 0.0f;
    for (int j = 0; j < k; ++j) {
        const int ej = __builtin_amdgcn_readlane(e, j);
        const float dj = uniform(dc, j);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (ej == lane + 64 * i) dp[i] += dj;
    }
    auto store = [&](auto value) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int x = lane + 64 * i;
            if (x < E) store_from_float<DT>(dlogits, t * E + x, value(i));
        }
    };
    if constexpr (SIGMOID) store([&](int i) { return dp[i] * pr[i]; });
    else if (renorm) store([&](int i) { return dp[i] + 0.0f * pr[i]; });  // (the row's NaN shows)
    else store([&](int i) { return pr[i] * (dp[i] - dot); });
}

template <int DT, int V>
hipError_t route_v(const RouteArgs &a, int log_lanes, hipStream_t s) {
    const bool keys = a.bias || (a.groups > 1 && a.group_top > 1);
    const dim3 grid((unsigned)((a.T + kWaves - 1) / kWaves)), block(kWaves * 64);
    if (keys && a.sigmoid) route_kernel<DT, V, true, true><<<grid, block, 0, s>>>(a, log_lanes);
    else if (keys) route_kernel<DT, V, true, false><<<grid, block, 0, s>>>(a, log_lanes);
    else if (a.sigmoid) route_kernel<DT, V, false, true><<<grid, block, 0, s>>>(a, log_lanes);
    else route_kernel<DT, V, false, false><<<grid, block, 0, s>>>(a, log_lanes);
    return hipGetLastError();
}

// Tokens of one launch: a grid holds fewer than 2^32 work items, 64 a token.
constexpr int64_t kMaxTokens = (int64_t)1 << 25;

template <int DT>
hipError_t route(RouteArgs a, hipStream_t s) {
    a.n = a.E / a.groups;
    int log_lanes = 6;  // the most lanes that 64 have for each group
    while ((a.groups << log_lanes) > 64) --log_lanes;
    const int own = (a.n + (1 << log_lanes) - 1) >> log_lanes;  // at most 31 for 1024 experts
    if (own <= 1) return route_v<DT, 1>(a, log_lanes, s);
    if (own <= 2) return route_v<DT, 2>(a, log_lanes, s);
    if (own <= 4) return route_v<DT, 4>(a, log_lanes, s);
    if (own <= 8) return route_v<DT, 8>(a, log_lanes, s);
    return route_v<DT, 32>(a, log_lanes, s);
}

template <int DT, int V>
hipError_t backward_v(const void *l, const int32_t *idx, const float *dw, void *dl, int64_t T, int E, int k, bool sigmoid,
                      bool renorm, hipStream_t s) {
    const dim3 grid((unsigned)((T + kWaves - 1) / kWaves)), block(kWaves * 64);
    if (sigmoid) route_backward_kernel<DT, V, true><<<grid, block, 0, s>>>(l, idx, dw, dl, T, E, k, renorm);
    else route_backward_kernel<DT, V, false><<<grid, block, 0, s>>>(l, idx, dw, dl, T, E, k, renorm);
    return hipGetLastError();
}

template <int DT>
hipError_t backward(const void *l, const int32_t *idx, const float *dw, void *dl, int64_t T, int E, int k, bool sigmoid,
                    bool renorm, hipStream_t s) {
    if (E <= 64) return backward_v<DT, 1>(l, idx, dw, dl, T, E, k, sigmoid, renorm, s);
    if (E <= 128) return backward_v<DT, 2>(l, idx, dw, dl, T, E, k, sigmoid, renorm, s);
    if (E <= 256) return backward_v<DT, 4>(l, idx, dw, dl, T, E, k, sigmoid, renorm, s);
    return backward_v<DT, 16>(l, idx, dw, dl, T, E, k, sigmoid, renorm, s);
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs &all, hipStream_t s) {
    hipError_t e = hipSuccess;
    for (int64_t t = 0; t < all.T && e == hipSuccess; t += kMaxTokens) {
        RouteArgs a = all;
        a.logits = static_cast<const char *>(all.logits) + t * all.E * (all.dtype == kF32 ? 4 : 2);
        a.idx += t * all.k, a.weights += t * all.k;
        a.T = all.T - t < kMaxTokens ? all.T - t : kMaxTokens;
        e = all.dtype == kF32 ? route<kF32>(a, s) : all.dtype == kF16 ? route<kF16>(a, s) : route<kBF16>(a, s);
    }
    return e;
}

hipError_t launch_moe_route_backward(const void *logits, const int32_t *idx, const float *dw, void *dlogits, int64_t T,
                                     int E, int k, int dtype, bool sigmoid, bool renorm, hipStream_t s) {
    hipError_t e = hipSuccess;
    for (int64_t t = 0; t < T && e == hipSuccess; t += kMaxTokens) {
        const int64_t n = T - t < kMaxTokens ? T - t : kMaxTokens, at = t * E * (dtype == kF32 ? 4 : 2);
        const void *l = static_cast<const char *>(logits) + at;
        void *dl = static_cast<char *>(dlogits) + at;
        const int32_t *i = idx + t * k;
        const float *d = dw + t * k;
        if (dtype == kF32) e = backward<kF32>(l, i, d, dl, n, E, k, sigmoid, renorm, s);
        else if (dtype == kF16) e = backward<kF16>(l, i, d, dl, n, E, k, sigmoid, renorm, s);
        else e = backward<kBF16>(l, i, d, dl, n, E, k, sigmoid, renorm, s);
    }
    return e;
}

}  // namespace tq2
