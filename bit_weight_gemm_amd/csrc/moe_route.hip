// A mixture's router: scores, groups, the k chosen experts and their weights, and
// the gradient of the weights with respect to the logits.
//
// Score p_e = softmax(l)_e or sigmoid(l_e); an expert's key is its logit (no bias and
// no sum of several keys per group: softmax and sigmoid are monotonic), else p_e +
// bias_e.  A group's key is the sum of its group_top best keys; the `keep` best groups
// stay.  Among what is left the k largest keys are chosen, the first at slot 0; equal
// keys go to the lower index.  weights[j] = p of slot j's expert, divided by the sum
// over the slots if renorm.
//
// A logit of -inf masks its expert (so does a bias of -inf, or a dropped group):
// it is never chosen, and slots that find no expert get idx -1 and weight 0, which
// the experts' products skip.  A NaN logit ranks first, so that it shows.
//
// Keys that are sums are formed and compared in f64: near ties decide whole numbers,
// and over 16384 tokens of 256 experts f32 scores swap a pair every few calls.
//
// One wave per token, lane l holding the experts l, l + 64, ... .  The k passes over
// the keys compare their f32 roundings (monotonic in the key) by a wave maximum in
// DPP; only when several keys share the largest rounding are the f64 values looked at.
#include <type_traits>

#include "q4.h"

namespace tq2 {

namespace {

constexpr int kWaves = 4;  // tokens per workgroup

__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp<0xB1>(v));
    v = fmaxf(v, dpp<0x4E>(v));
    v = fmaxf(v, dpp<0x124>(v));
    v = fmaxf(v, dpp<0x128>(v));
    float a = v, b = v;
    swap16(a, b);
    v = fmaxf(a, b);
    a = v, b = v;
    swap32(a, b);
    return fmaxf(a, b);
}

__device__ __forceinline__ float wave_sum(float v) {
    v = row16_sum(v);
    float a = v, b = v;
    swap16(a, b);
    v = a + b;
    a = v, b = v;
    swap32(a, b);
    return a + b;
}

__device__ __forceinline__ double wave_sum(double v) {
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
    return v;
}

__device__ __forceinline__ double wave_max(double v) {
    for (int o = 1; o < 64; o <<= 1) {
        const double b = __shfl_xor(v, o);
        v = b > v ? b : v;
    }
    return v;
}

__device__ __forceinline__ double uniform(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ float uniform(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

constexpr float kNone = -__builtin_inff();

// V: experts per lane.  KEYS: keys are sums of scores (f64), else the logits.
template <int DT, int V, bool KEYS, bool SIGMOID>
__global__ __launch_bounds__(kWaves * 64) void route_kernel(RouteArgs p) {
    typedef typename std::conditional<KEYS, double, float>::type F;
    __shared__ F keys[kWaves][V * 64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= p.T) return;  // no barrier below: each wave uses its own LDS
    const int E = p.E;

    float l[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        l[i] = e < E ? load_as_float<DT>(p.logits, t * E + e) : kNone;
    }
    F score[V], key[V];
    F most = kNone, total = 1;
    if constexpr (!SIGMOID) {
        float m = kNone;
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
        most = wave_max(m);
        total = 0;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if constexpr (SIGMOID) score[i] = (F)1 / ((F)1 + exp(-(F)l[i]));
        else {
            score[i] = l[i] == kNone ? (F)0 : exp((F)l[i] - most);
            total += score[i];
        }
    }
    if constexpr (!SIGMOID) {
        total = wave_sum(total);
#pragma unroll
        for (int i = 0; i < V; ++i) score[i] /= total;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        key[i] = KEYS ? score[i] : (F)l[i];
        if (KEYS && p.bias && e < E) key[i] += (F)p.bias[e];
        if (l[i] == kNone) key[i] = kNone;
        if (key[i] != key[i]) key[i] = __builtin_inff();
    }
    if (p.groups > 1) {
        const int n = E / p.groups;
#pragma unroll
        for (int i = 0; i < V; ++i) keys[wave][lane + 64 * i] = key[i];
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // lane g: the best two keys of group g, starting at another place in each
        // group so that the lanes read different banks
        F a = kNone, b = kNone;
        if (lane < p.groups) {
            int at = lane % n;
            for (int i = 0; i < n; ++i) {
                const F v = keys[wave][lane * n + at];
                if (v > a) b = a, a = v;
                else if (v > b) b = v;
                if (++at == n) at = 0;
            }
            if (p.group_top > 1 && n > 1) a = b == kNone ? a : a + b;
        }
        // its place: the groups that beat it
        int place = 0;
        for (int g = 0; g < p.groups; ++g) {
            const F v = uniform(a, g);
            if (v > a || (v == a && g < lane)) ++place;
        }
        const uint64_t kept = __ballot(lane < p.groups && place < p.keep);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            if (e < E && !((kept >> (e / n)) & 1)) key[i] = kNone;
        }
    }
    float hi[V];
#pragma unroll
    for (int i = 0; i < V; ++i) hi[i] = (float)key[i];

    int mine = -1;
    F w = 0, sum = 0;
    for (int j = 0; j < p.k; ++j) {
        float m = hi[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = fmaxf(m, hi[i]);
        m = wave_max(m);
        if (m == kNone) break;
        // the experts whose key rounds to the maximum
        uint64_t at[V];
        int many = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            at[i] = __ballot(hi[i] == m);
            many += __popcll(at[i]);
        }
        if (KEYS && many > 1) {
            F top = kNone;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (hi[i] == m && key[i] > top) top = key[i];
            top = wave_max(top);
#pragma unroll
            for (int i = 0; i < V; ++i) at[i] = __ballot(hi[i] == m && key[i] == top);
        }
        int e = 0;
        F s = 0;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            if (at[i]) {
                const int at_lane = __builtin_ctzll(at[i]);
                e = 64 * i + at_lane;
                s = uniform(score[i], at_lane);
            }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e == lane + 64 * i) hi[i] = kNone;
        sum += s;
        if (lane == j) mine = e, w = s;
    }
    if (p.renorm && sum != 0) w /= sum;
    if (lane < p.k) {
        p.idx[t * p.k + lane] = mine;
        p.weights[t * p.k + lane] = (float)w;
    }
}

// dlogits of one token: with c_j the chosen scores, dc_j = dw_j, or with renorm
// (dw_j - sum_i dw_i c_i / sum c) / sum c; then dp scattered to the experts and
// through softmax dl = p (dp - sum dp p), or sigmoid dl = dp p (1 - p).
template <int DT, int V, bool SIGMOID>
__global__ __launch_bounds__(kWaves * 64) void route_backward_kernel(const void *logits, const int32_t *idx, const float *dw,
                                                                     void *dlogits, int64_t T, int E, int k, int renorm) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= T) return;
    int e = -1;
    float dc = 0.0f, c = 0.0f;
    if (lane < k) {
        e = idx[t * k + lane];
        if (e < 0 || e >= E) e = -1;
        else {
            dc = dw[t * k + lane];
            c = load_as_float<DT>(logits, t * E + e);
        }
    }
    float l[V], pr[V];
    float most = kNone;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int x = lane + 64 * i;
        l[i] = x < E ? load_as_float<DT>(logits, t * E + x) : kNone;
        most = fmaxf(most, l[i]);
    }
    if constexpr (SIGMOID) {
#pragma unroll
        for (int i = 0; i < V; ++i) pr[i] = 1.0f / (1.0f + expf(-l[i]));
        c = 1.0f / (1.0f + expf(-c));
    } else {
        most = wave_max(most);
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) total += pr[i] = l[i] == kNone ? 0.0f : expf(l[i] - most);
        total = wave_sum(total);
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;  // 0: every logit is -inf
#pragma unroll
        for (int i = 0; i < V; ++i) pr[i] *= inv;
        c = c == kNone ? 0.0f : expf(c - most) * inv;
    }
    if (e < 0) c = 0.0f;
    float dot = wave_sum(dc * c);
    if (renorm) {
        const float total = wave_sum(c);
        dc = e < 0 || total == 0.0f ? 0.0f : (dc - dot / total) / total;
        dot = wave_sum(dc * c);
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
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int x = lane + 64 * i;
        const float v = SIGMOID ? dp[i] * pr[i] * (1.0f - pr[i]) : pr[i] * (dp[i] - dot);
        if (x < E) store_from_float<DT>(dlogits, t * E + x, v);
    }
}

template <int DT, int V>
hipError_t route_v(const RouteArgs &a, hipStream_t s) {
    const bool keys = a.bias || (a.groups > 1 && a.group_top > 1);
    const dim3 grid((unsigned)((a.T + kWaves - 1) / kWaves)), block(kWaves * 64);
    if (keys && a.sigmoid) route_kernel<DT, V, true, true><<<grid, block, 0, s>>>(a);
    else if (keys) route_kernel<DT, V, true, false><<<grid, block, 0, s>>>(a);
    else if (a.sigmoid) route_kernel<DT, V, false, true><<<grid, block, 0, s>>>(a);
    else route_kernel<DT, V, false, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t route(const RouteArgs &a, hipStream_t s) {
    if (a.E <= 64) return route_v<DT, 1>(a, s);
    if (a.E <= 128) return route_v<DT, 2>(a, s);
    if (a.E <= 256) return route_v<DT, 4>(a, s);
    return route_v<DT, 16>(a, s);
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

hipError_t launch_moe_route(const RouteArgs &a, hipStream_t s) {
    if (a.dtype == kF32) return route<kF32>(a, s);
    if (a.dtype == kF16) return route<kF16>(a, s);
    return route<kBF16>(a, s);
}

hipError_t launch_moe_route_backward(const void *logits, const int32_t *idx, const float *dw, void *dlogits, int64_t T,
                                     int E, int k, int dtype, bool sigmoid, bool renorm, hipStream_t s) {
    if (dtype == kF32) return backward<kF32>(logits, idx, dw, dlogits, T, E, k, sigmoid, renorm, s);
    if (dtype == kF16) return backward<kF16>(logits, idx, dw, dlogits, T, E, k, sigmoid, renorm, s);
    return backward<kBF16>(logits, idx, dw, dlogits, T, E, k, sigmoid, renorm, s);
}

}  // namespace tq2
