// A whole mixture-of-experts layer: n = norm(x), logits = n router^T, the router's choice, the experts' products, the residual.
//
// The logits decide which experts a token has.  They are summed in f64 and rounded to f32, so that the choice does not
// depend on how many tokens a call has or on how their sums are dealt to threads.
#include "moe_layer.h"

#include "block_norm.h"
#include "moe_route.h"

namespace tq2 {

namespace {

// Tokens times experts up to which the norm and the logits are one launch, whose workgroups norm a row again for every four experts.
// Norm and logits in one launch / apart, bf16 rows, f32 router, us: 64 experts, d = 2048, 64 tokens 7.3 / 8.6, 128 9.7 / 9.6, 256 16 / 14,
// 512 25 / 18; 256 experts, 16 tokens 6.3 / 7.5, 32 10.3 / 10.2, 64 17 / 15; 8 experts, d = 1024, 512 tokens 6.3 / 8.0, 1024 10.6 / 10.0.
constexpr int64_t kNormWithLogits = 8192;
// And up to which a workgroup without a norm has four experts, beyond eight.  Layers with four / eight, f32 router, us: 128 tokens of 128
// experts, d = 4096, 61 / 63, 256 of them 80 / 82; 2048 of 64, d = 2048, 111 / 110, 1024 of 256 183 / 178 (bf16 router 190 / 184).
constexpr int64_t kLogitsOfFour = 32768;

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
    // One expert to a workgroup while the chip has room for them, then four, then eight (2048 tokens of 64 experts, d = 2048,
    // bf16, f32 router: norm and logits 64 us).
    const dim3 block(256);
    if ((int64_t)a.T * a.E <= 1024) layer_logits_kernel<DT, WT, RT, NORM, 1><<<dim3(a.E, a.T), block, 0, s>>>(a);
    else if (NORM || (int64_t)a.T * a.E <= kLogitsOfFour) layer_logits_kernel<DT, WT, RT, NORM, 4><<<dim3((a.E + 3) / 4, a.T), block, 0, s>>>(a);
    else if constexpr (!NORM) layer_logits_kernel<DT, WT, RT, NORM, 8><<<dim3((a.E + 7) / 8, a.T), block, 0, s>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t logits_of(const LogitsArgs &a, bool wide_norm, bool wide_router, hipStream_t s) {
    if constexpr (DT == kF32) {
        return a.norm ? logits_of<DT, DT, DT, true>(a, s) : logits_of<DT, DT, DT, false>(a, s);
    } else {
        if (!a.norm) return wide_router ? logits_of<DT, DT, kF32, false>(a, s) : logits_of<DT, DT, DT, false>(a, s);
        if (wide_norm) return wide_router ? logits_of<DT, kF32, kF32, true>(a, s) : logits_of<DT, kF32, DT, true>(a, s);
        return wide_router ? logits_of<DT, DT, kF32, true>(a, s) : logits_of<DT, DT, DT, true>(a, s);
    }
}

// All tokens', as many at a time as a grid's second axis has.
hipError_t launch_logits(LogitsArgs l, int64_t T, int dtype, bool wide_norm, bool wide_router, hipStream_t s) {
    constexpr int64_t kMost = 65535;
    const size_t row = (size_t)l.d * (dtype == kF32 ? 4 : 2);
    hipError_t e = hipSuccess;
    for (int64_t t = 0; t < T && e == hipSuccess; t += kMost) {
        l.T = (int)(T - t < kMost ? T - t : kMost);
        if (dtype == kF32) e = logits_of<kF32>(l, wide_norm, wide_router, s);
        else if (dtype == kF16) e = logits_of<kF16>(l, wide_norm, wide_router, s);
        else e = logits_of<kBF16>(l, wide_norm, wide_router, s);
        l.x = static_cast<const char *>(l.x) + kMost * row, l.logits += kMost * l.E;
    }
    return e;
}

// One launch behind the logits' for a token or two, and for up to four of eight slots and more, where the weights have groups of 128.
// Together / apart (choice, two products), us of graph replays with norm and residual, zero points or not within 3%:
//                                       bf16: one token    two          three        four         f32: one     two          four
//   64 experts of 8, 2048 x 1024        19.5 / 19.9        22.8 / 23.9  27.9 / 30.2  31.8 / 33.0  24.0 / 24.6  29.4 / 30.8  46.0 / 45.0
//   128 of 8, 2048 x 768                18.3 / 18.5        22.7 / 22.0  25.2 / 29.3  27.9 / 30.2  22.7 / 22.5  28.0 / 28.5  37.1 / 39.4
//   32 of 16, 2048 x 512                19.9 / 20.3        23.6 / 23.2  (above 32 slots)          23.9 / 24.6  29.3 / 30.1
//   64 of 4, 1024 x 1024                13.8 / 14.6        14.5 / 15.2                            15.4 / 16.8  16.6 / 17.6
//   8 of 2, 1024 x 1024                 11.9 / 11.9        12.4 / 12.1                            13.1 / 13.6  13.5 / 13.8
// With a host in front of each call the small ones are 12.1 / 15.4 and 12.6 / 15.8 (8 of 2): it has one launch less to make.  Four tokens
// of 64 of 2 18.4 / 17.5, eight of 8 57 / 51.  With groups of 32 and 64 the one launch kept up to 336 bytes a lane in scratch and
// lost: 64 of 8, one token 39 / 21 and 24 / 20, four 81 / 35 and 41 / 33 (f32, 32: 46 / 25 and 98 / 52).
bool few_tokens(int64_t T, int64_t k) { return T * k <= 32 && (T <= 2 || k >= 8); }

}  // namespace

LayerPlan layer_plan(int64_t T, int64_t k, int64_t E, int64_t groups, int64_t d, int64_t f, int dtype, bool norm, bool coarse) {
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    LayerPlan p{};
    p.moe = moe_plan(T, k, E, d, f, dtype);
    p.few = coarse && p.moe.direct && few_tokens(T, k) && T * E <= kNormWithLogits && route_own((int)E, (int)groups) <= kFewOwn;
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
    LogitsArgs l{};
    l.x = a.x, l.norm = a.norm, l.router = a.router, l.n = b, l.logits = logits, l.eps = a.eps, l.E = E, l.d = d;
    if (a.norm && a.T * E > kNormWithLogits) {  // the norm in a launch of its own, once for all experts
        BlockNormArgs q{};
        q.x = a.x, q.pre = a.norm, q.n = b, q.M = a.T, q.gate_rows = a.T, q.N = d, q.eps = a.eps, q.scale = 1.0f;
        e = launch_block_norm(q, a.dtype, a.wide_norm, s);
        if (e != hipSuccess) return e;
        l.x = n, l.norm = nullptr;
    }
    char *h = b + p.off_moe + p.moe.off_h;
    if (p.few) {
        l.fill = reinterpret_cast<w4 *>(h), l.fill_rows = a.route.k * (a.dtype == kF32 ? 3 : 2);
        l.fill_pitch = (int)(p.moe.ldh / 8), l.fill_own = a.gate.N / 8;
    }
    e = launch_logits(l, a.T, a.dtype, a.wide_norm, a.wide_router, s);
    if (e != hipSuccess) return e;
    if (p.few) return launch_few_experts(FewArgs{n, logits, h, patience}, a, s);
    RouteArgs r = a.route;
    r.logits = logits, r.dtype = kF32;
    e = launch_moe_route(r, s);
    if (e != hipSuccess) return e;
    return launch_q4_moe(p.moe, n, r.idx, r.weights, a.gate, a.up, a.down, a.residual, a.y, a.T, r.k, a.dtype, b + p.off_moe, s);
}

}  // namespace tq2
