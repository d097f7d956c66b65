// A whole mixture-of-experts layer: n = norm(x), logits = n router^T, the router's choice, the experts' products, the residual.
//
// The logits decide which experts a token has.  They are summed in f64 and rounded to f32, so that the choice does not
// depend on how many tokens a call has or on how their sums are dealt to threads.
#include "moe_layer.h"

#include "block_norm.h"

namespace tq2 {

namespace {

// One wave per token and expert.
template <int DT, int RT>
__global__ __launch_bounds__(256) void layer_logits_kernel(const void *x, const void *router, float *logits, int64_t T, int E, int d) {
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
void logits_of(const void *x, const void *router, float *logits, int64_t T, int E, int d, hipStream_t s) {
    layer_logits_kernel<DT, RT><<<dim3((unsigned)((T * E + 3) / 4)), dim3(256), 0, s>>>(x, router, logits, T, E, d);
}

}  // namespace

LayerPlan layer_plan(int64_t T, int64_t k, int64_t E, int64_t d, int64_t f, int dtype, bool norm) {
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    LayerPlan p{};
    p.moe = moe_plan(T, k, E, d, f, dtype);
    p.off_logits = norm ? up((size_t)T * d * (dtype == kF32 ? 4 : 2)) : 0;
    p.off_moe = p.off_logits + up((size_t)T * E * 4);
    p.total = p.off_moe + p.moe.total;
    return p;
}

hipError_t launch_moe_layer(const LayerPlan &p, const LayerArgs &a, void *ws, hipStream_t s) {
    char *b = static_cast<char *>(ws);
    const int d = a.gate.K, E = a.gate.E;
    const void *n = a.x;
    hipError_t e;
    if (a.norm) {
        BlockNormArgs q{};
        q.x = a.x, q.pre = a.norm, q.n = b, q.M = a.T, q.gate_rows = a.T, q.N = d, q.eps = a.eps, q.scale = 1.0f;
        e = launch_block_norm(q, a.dtype, a.wide_norm, s);
        if (e != hipSuccess) return e;
        n = b;
    }
    float *logits = reinterpret_cast<float *>(b + p.off_logits);
    if (a.dtype == kF32) logits_of<kF32, kF32>(n, a.router, logits, a.T, E, d, s);
    else if (a.dtype == kF16 && a.wide_router) logits_of<kF16, kF32>(n, a.router, logits, a.T, E, d, s);
    else if (a.dtype == kF16) logits_of<kF16, kF16>(n, a.router, logits, a.T, E, d, s);
    else if (a.wide_router) logits_of<kBF16, kF32>(n, a.router, logits, a.T, E, d, s);
    else logits_of<kBF16, kBF16>(n, a.router, logits, a.T, E, d, s);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    RouteArgs r = a.route;
    r.logits = logits, r.dtype = kF32;
    e = launch_moe_route(r, s);
    if (e != hipSuccess) return e;
    return launch_q4_moe(p.moe, n, r.idx, r.weights, a.gate, a.up, a.down, a.residual, a.y, a.T, r.k, a.dtype, b + p.off_moe, s);
}

}  // namespace tq2
