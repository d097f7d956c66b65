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
#include "moe_route.h"

namespace tq2 {

namespace {

constexpr int kWaves = 4;  // tokens per workgroup

// V: experts per lane.  KEYS: keys are sums of scores, else the logits.
template <int DT, int V, bool KEYS, bool SIGMOID>
__global__ __launch_bounds__(kWaves * 64) void route_kernel(RouteArgs p, int log_lanes) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= p.T) return;
    const Place at = route_place(p, log_lanes, lane);
    float l[V], key[V];  // key: of the biases first
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i < at.own ? at.first + i * at.lanes : 0;
        l[i] = load_as_float<DT>(p.logits, t * p.E + e);
        key[i] = KEYS && p.bias ? p.bias[e] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = i < at.own ? l[i] : kNone;
    float most, total;
    const int mine = route_choose<V, KEYS, SIGMOID>(p, l, key, at, log_lanes, lane, true, most, total);
    const float chosen = load_as_float<DT>(p.logits, t * p.E + (mine < 0 ? 0 : mine));
    const float w = route_weight<SIGMOID>(p, mine, chosen, most, total);
    if (lane < p.k) {
        p.idx[t * p.k + lane] = mine;
        p.weights[t * p.k + lane] = w;
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
