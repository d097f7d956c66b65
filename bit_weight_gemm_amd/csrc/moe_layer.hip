// A whole mixture-of-experts layer: n = norm(x), logits = n router^T, the router's choice, the experts' products, the residual.
//
// The logits decide which experts a token has.  They are summed in f64 and rounded to f32, so that the choice does not
// depend on how many tokens a call has or on how their sums are dealt to threads.
#include "moe_layer.h"

#include "block_norm.h"
#include "moe_route.h"

namespace tq2 {

namespace {

struct LogitsArgs {
    const void *x, *norm, *router;
    void *n;                 // NORM: [T][d]
    float *logits;
    w4 *fill;                // [T fill_rows][fill_pitch] pieces of 0xff bytes, of 0 from fill_own on
    int fill_rows, fill_pitch, fill_own;
    double eps;
    int T, E, d;
};

// One token and EB experts to a workgroup: the row is normed (every workgroup of a token does; the first keeps the result), and multiplied
// with EB rows of the router.  A thread has eight columns of each 2048; the first ones' loads are all sent at once.
template <int DT, int WT, int RT, bool NORM, int EB>
__global__ __launch_bounds__(256) void layer_logits_kernel(LogitsArgs p) {
    __shared__ double room[2][4 * EB];
    const int tid = threadIdx.x, d = p.d, e0 = blockIdx.x * EB;
    const int64_t t = blockIdx.y;
    Raw<DT, 8> x;
    Raw<WT, 8> w;
    Raw<RT, 8> r[EB];
    auto load = [&](int k0) {
        const Piece<8, kWhole> at((k0 >> 3) + tid, d);
        at.template load<DT>(p.x, t * d, d, x);
        if constexpr (NORM) at.template load<WT>(p.norm, 0, d, w);
#pragma unroll
        for (int q = 0; q < EB; ++q) at.template load<RT>(p.router, (int64_t)(e0 + q < p.E ? e0 + q : e0) * d, d, r[q]);
    };
    load(0);
    for (int row = blockIdx.x; row < p.fill_rows; row += gridDim.x)
        for (int i = tid; i < p.fill_pitch; i += 256)
            p.fill[(t * p.fill_rows + row) * p.fill_pitch + i] = i < p.fill_own ? ~w4{} : w4{};
    Norm norm{};
    if constexpr (NORM) {
        double sum[1] = {};
        for (int k0 = 0; k0 < d; k0 += 2048) {
            const Piece<8, kWhole> at((k0 >> 3) + tid, d);
            Raw<DT, 8> raw = x;
            if (k0) at.template load<DT>(p.x, t * d, d, raw);
            float v[8];
            at.template values<DT>(raw, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) sum[0] += (double)v[q] * v[q];
        }
        row_total<256, 1>(sum, room[0]);
        norm = norm_of(0.0, sum[0], d, false, p.eps);
    }
    double dot[EB] = {};
    for (int k0 = 0; k0 < d; k0 += 2048) {
        const Piece<8, kWhole> at((k0 >> 3) + tid, d);
        if (k0) load(k0);
        float v[8];
        at.template values<DT>(x, v);
        if constexpr (NORM) {
            float k[8];
            at.template values<WT>(w, k);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = rounded<DT>(norm_value<false>(norm, v[q], k[q], 0.0f));
            if (blockIdx.x == 0 && at.any()) at.template store<DT>(p.n, t * d, v);
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) {
            float k[8];
            at.template values<RT>(r[e], k);
#pragma unroll
            for (int q = 0; q < 8; ++q) dot[e] += (double)v[q] * k[q];
        }
    }
    row_total<256, EB>(dot, room[1]);
#pragma unroll
    for (int e = 0; e < EB; ++e)
        if (tid == e && e0 + e < p.E) p.logits[t * p.E + e0 + e] = (float)dot[e];
}

template <int DT, int WT, int RT, bool NORM>
hipError_t logits_of(const LogitsArgs &a, hipStream_t s) {
    // one expert to a workgroup while the chip has room for them, then four
    if ((int64_t)a.T * a.E <= 1024) layer_logits_kernel<DT, WT, RT, NORM, 1><<<dim3(a.E, a.T), dim3(256), 0, s>>>(a);
    else layer_logits_kernel<DT, WT, RT, NORM, 4><<<dim3((a.E + 3) / 4, a.T), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t logits_of(const LogitsArgs &a, bool wide_norm, bool wide_router, hipStream_t s) {
    if (!a.norm) return wide_router ? logits_of<DT, DT, kF32, false>(a, s) : logits_of<DT, DT, DT, false>(a, s);
    if (wide_norm) return wide_router ? logits_of<DT, kF32, kF32, true>(a, s) : logits_of<DT, kF32, DT, true>(a, s);
    return wide_router ? logits_of<DT, DT, kF32, true>(a, s) : logits_of<DT, DT, DT, true>(a, s);
}

// One wave per token and expert.
template <int DT, int RT>
__global__ __launch_bounds__(256) void prompt_logits_kernel(const void *x, const void *router, float *logits, int64_t T, int E, int d) {
    const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (at >= T * E) return;
    const int64_t t = at / E, e = at % E;
    double sum = 0.0;
    for (int k = lane; k < d; k += 64) sum += (double)load_as_float<DT>(x, t * d + k) * load_as_float<RT>(router, e * d + k);
    sum = wave_total(sum);
    if (lane == 0) logits[at] = (float)sum;
}

template <int DT, int RT>
void prompt_logits(const void *x, const void *router, float *logits, int64_t T, int E, int d, hipStream_t s) {
    prompt_logits_kernel<DT, RT><<<dim3((unsigned)((T * E + 3) / 4)), dim3(256), 0, s>>>(x, router, logits, T, E, d);
}

// Up to so many slots the experts' choice and products are one launch (64 experts of 8, 2048 x 1024, bf16: one token 17.4 us, two 23,
// four 31.6; the choice and the two products apart, four 32.9, eight 51 against 57).
constexpr int64_t kFewMost = 32;
// Tokens times experts up to which the norm and the logits are one launch.
constexpr int64_t kLogitsSmall = 32768;

}  // namespace

LayerPlan layer_plan(int64_t T, int64_t k, int64_t E, int64_t groups, int64_t d, int64_t f, int dtype, bool norm) {
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    LayerPlan p{};
    p.moe = moe_plan(T, k, E, d, f, dtype);
    p.few = p.moe.direct && T * k <= kFewMost && T * E <= kLogitsSmall && route_own((int)E, (int)groups) <= kFewOwn;
    p.off_logits = norm ? up((size_t)T * d * (dtype == kF32 ? 4 : 2)) : 0;
    p.off_moe = p.off_logits + up((size_t)T * E * 4);
    p.total = p.off_moe + p.moe.total;
    return p;
}

hipError_t launch_moe_layer(const LayerPlan &p, const LayerArgs &a, void *ws, int patience, hipStream_t s) {
    char *b = static_cast<char *>(ws);
    const int d = a.gate.K, E = a.gate.E;
    float *logits = reinterpret_cast<float *>(b + p.off_logits);
    const void *n = a.norm ? b : a.x;
    hipError_t e;
    if (a.T * E <= kLogitsSmall) {  // with the norm, in one launch
        LogitsArgs l{};
        l.x = a.x, l.norm = a.norm, l.router = a.router, l.n = b, l.logits = logits, l.eps = a.eps;
        l.T = (int)a.T, l.E = E, l.d = d;
        char *h = b + p.off_moe + p.moe.off_h;
        if (p.few) {
            l.fill = reinterpret_cast<w4 *>(h), l.fill_rows = a.route.k * (a.dtype == kF32 ? 3 : 2);
            l.fill_pitch = (int)(p.moe.ldh / 8), l.fill_own = a.gate.N / 8;
        }
        if (a.dtype == kF32) e = a.norm ? logits_of<kF32, kF32, kF32, true>(l, s) : logits_of<kF32, kF32, kF32, false>(l, s);
        else if (a.dtype == kF16) e = logits_of<kF16>(l, a.wide_norm, a.wide_router, s);
        else e = logits_of<kBF16>(l, a.wide_norm, a.wide_router, s);
        if (e != hipSuccess) return e;
        if (p.few) return launch_few_experts(FewArgs{n, logits, h, patience}, a, s);
    } else {
        if (a.norm) {
            BlockNormArgs q{};
            q.x = a.x, q.pre = a.norm, q.n = b, q.M = a.T, q.gate_rows = a.T, q.N = d, q.eps = a.eps, q.scale = 1.0f;
            e = launch_block_norm(q, a.dtype, a.wide_norm, s);
            if (e != hipSuccess) return e;
        }
        if (a.dtype == kF32) prompt_logits<kF32, kF32>(n, a.router, logits, a.T, E, d, s);
        else if (a.dtype == kF16 && a.wide_router) prompt_logits<kF16, kF32>(n, a.router, logits, a.T, E, d, s);
        else if (a.dtype == kF16) prompt_logits<kF16, kF16>(n, a.router, logits, a.T, E, d, s);
        else if (a.wide_router) prompt_logits<kBF16, kF32>(n, a.router, logits, a.T, E, d, s);
        else prompt_logits<kBF16, kBF16>(n, a.router, logits, a.T, E, d, s);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    RouteArgs r = a.route;
    r.logits = logits, r.dtype = kF32;
    e = launch_moe_route(r, s);
    if (e != hipSuccess) return e;
    return launch_q4_moe(p.moe, n, r.idx, r.weights, a.gate, a.up, a.down, a.residual, a.y, a.T, r.k, a.dtype, b + p.off_moe, s);
}

}  // namespace tq2
