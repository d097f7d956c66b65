// A few tokens through a mixture's experts in one launch, from the router's logits: y[t] = residual[t] +
// sum_j w_j down_e(silu(gate_e n_t) * (up_e n_t)).
//
// The first T k gx workgroups have the slots' gate and up products (32 columns of one slot each), the others the down
// products (16 columns of one token each).  Each chooses its token's experts from the logits itself (one wave, against a
// launch of its own).  The down workgroups send the loads of their first codes and then read silu(g) u, which may not be there yet:
// the launch before has filled it with a pattern that no value has, and who reads the pattern reads again.  So nobody counts
// and nothing is fenced.  (384 tickets and 256 counts at one address took one token 34 us, fences at device scope, which write back
// and empty a whole L2 each, 52.)
//
// Every wait ends.  The gate and up workgroups wait for nobody, and the hardware starts workgroups in order; but should a down
// workgroup have waited `patience` times for a value, because those before it are not running, it gives up, forms its
// token's silu(g) u itself (the same values at the same places) and begins again.
#include "moe_layer.h"
#include "moe_route.h"
#include "q4_row.h"

namespace tq2 {

namespace {

constexpr int kFewWaves = 8, kFewSlots = 64;

// The argument block is read line by line, each from far: a call has no more of it than it needs, and all of it is asked for at once.
struct FewWeight {
    const w4 *codes;
    const uint16_t *scales;
    const uint8_t *zeros;
};
struct FewCall {
    FewWeight gate, up, down;
    const void *n, *residual;
    void *h, *y;
    const float *logits, *bias;
    int32_t *idx;
    float *weights;
    int E, d, f, T, k, gx, dx;  // gx, dx: workgroups of a slot, and of a token's down products
    int ldh, patience;
    int groups, keep, per_group, log_lanes;
    int flags;               // kFew...
};
enum { kFewSigmoid = 1, kFewRenorm = 2, kFewTopTwo = 4, kFewOne = 8 };  // kFewOne: a lane of the router has one expert at most

__device__ __forceinline__ Q4View few_view(const FewWeight &w, int E, int N, int K, int G) {
    Q4View v{};
    v.codes = w.codes, v.scales = w.scales, v.zeros = w.zeros, v.E = E, v.N = N, v.K = K, v.G = G;
    v.nb = (N + 15) >> 4, v.ku = (K + 127) >> 7;
    return v;
}

template <int XT, int XH, int G, int GD, int PH, int DT, bool RES>
__global__ __launch_bounds__(kFewWaves * 64, 4) void few_experts_kernel(FewCall p) {
    asm volatile("" ::"s"(p.gate.codes), "s"(p.gate.scales), "s"(p.gate.zeros), "s"(p.up.codes), "s"(p.up.scales), "s"(p.up.zeros),
                 "s"(p.down.codes), "s"(p.down.scales), "s"(p.down.zeros), "s"(p.n), "s"(p.residual), "s"(p.h), "s"(p.y),
                 "s"(p.logits), "s"(p.bias), "s"(p.idx), "s"(p.weights), "s"(p.E), "s"(p.d), "s"(p.f), "s"(p.T), "s"(p.k), "s"(p.gx),
                 "s"(p.dx), "s"(p.ldh), "s"(p.patience), "s"(p.groups), "s"(p.keep), "s"(p.log_lanes), "s"(p.flags));
    extern __shared__ __attribute__((aligned(16))) uint16_t few_room[];
    __shared__ float red[kFewWaves][64];
    __shared__ int32_t chosen[kFewSlots];
    __shared__ float weights[kFewSlots];
    const int tid = threadIdx.x, lane = tid & 63, k = p.k;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ups = p.T * k * p.gx, tasks = ups + p.T * p.dx;
    RouteArgs route{};
    route.bias = p.bias, route.E = p.E, route.k = k, route.groups = p.groups, route.keep = p.keep, route.n = p.per_group;
    route.group_top = p.flags & kFewTopTwo ? 2 : 1, route.sigmoid = p.flags & kFewSigmoid, route.renorm = p.flags & kFewRenorm;
    Q4RowArgs up{}, down{};
    up.w = few_view(p.gate, p.E, p.f, p.d, G), up.w2 = few_view(p.up, p.E, p.f, p.d, G);
    up.x = p.n, up.y = p.h, up.ldh = p.ldh, up.topk = k;
    down.w = few_view(p.down, p.E, p.d, p.f, GD);
    down.x = p.h, down.y = p.y, down.ldh = p.ldh, down.topk = k, down.residual = p.residual, down.patience = p.patience;
    // every wave chooses for every eighth token
    for (int t = wave; t < p.T; t += kFewWaves) {
        const float *logits = p.logits + (int64_t)t * p.E;
        const bool weigh = (int)blockIdx.x + (tasks - 1 - (int)blockIdx.x) / (int)gridDim.x * (int)gridDim.x >= ups;  // has a down task
        const Slot s = p.flags & kFewOne ? route_token<1>(route, logits, p.log_lanes, lane, weigh)
                             : route_token<kFewOwn>(route, logits, p.log_lanes, lane, weigh);
        if (lane < k) {
            const int at = t * k + lane;
            chosen[at] = s.expert, weights[at] = s.weight;
            if (blockIdx.x == gridDim.x - 1) p.idx[at] = s.expert, p.weights[at] = s.weight;  // (has the last task)
        }
    }
    __syncthreads();
    float(*red16)[16] = reinterpret_cast<float(*)[16]>(&red[0][0]);
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
        const bool is_up = task < ups;
        const int at = task - ups, t = is_up ? 0 : at / p.dx;
        for (bool form = is_up;; form = true) {
            if (form) {
                const int first = is_up ? task : t * k * p.gx, last = is_up ? task + 1 : (t + 1) * k * p.gx;
                for (int i = first; i < last; ++i) {
                    const int slot = i / p.gx;
                    q4_row_task<XT, G, 4, kFewWaves, 2, kRowGateUp, PH, kF32, false, true>(
                        up, i % p.gx, slot, Q4Slots{chosen + slot, weights + slot}, few_room, red);
                    __syncthreads();  // the rooms are free again
                }
                if (is_up) break;
            }
            const bool done = q4_row_task<XH, GD, 1, kFewWaves, 8, kRowDownSum, 1, DT, RES, true>(
                down, at % p.dx, t, Q4Slots{chosen + t * k, weights + t * k}, few_room, red16);
            __syncthreads();
            if (done) break;
        }
    }
}

template <int XT, int XH, int PH, int DT, int G, int GD>
hipError_t run(const FewCall &c, size_t lds, bool residual, hipStream_t s) {
    // two workgroups to each of the 256 compute units, if there is work for them
    const int tasks = c.T * (c.k * c.gx + c.dx);
    const dim3 grid((unsigned)(tasks < 512 ? tasks : 512)), block(kFewWaves * 64);
    if (residual) few_experts_kernel<XT, XH, G, GD, PH, DT, true><<<grid, block, lds, s>>>(c);
    else few_experts_kernel<XT, XH, G, GD, PH, DT, false><<<grid, block, lds, s>>>(c);
    return hipGetLastError();
}

template <int XT, int XH, int PH, int DT, int G>
hipError_t run(const FewCall &c, int gd, size_t lds, bool residual, hipStream_t s) {
    if (gd == 32) return run<XT, XH, PH, DT, G, 32>(c, lds, residual, s);
    if (gd == 64) return run<XT, XH, PH, DT, G, 64>(c, lds, residual, s);
    return run<XT, XH, PH, DT, G, 128>(c, lds, residual, s);
}

template <int XT, int XH, int PH, int DT>
hipError_t run(const FewCall &c, const LayerArgs &a, size_t lds, hipStream_t s) {
    const bool residual = a.residual != nullptr;
    if (a.gate.G == 32) return run<XT, XH, PH, DT, 32>(c, a.down.G, lds, residual, s);
    if (a.gate.G == 64) return run<XT, XH, PH, DT, 64>(c, a.down.G, lds, residual, s);
    return run<XT, XH, PH, DT, 128>(c, a.down.G, lds, residual, s);
}

}  // namespace

hipError_t launch_few_experts(const FewArgs &f, const LayerArgs &a, hipStream_t s) {
    const RouteArgs &r = a.route;
    auto weight = [](const Q4View &v) { return FewWeight{v.codes, v.scales, v.zeros}; };
    FewCall c{};
    c.gate = weight(a.gate), c.up = weight(a.up), c.down = weight(a.down);
    c.n = f.n, c.residual = a.residual, c.h = f.h, c.y = a.y, c.logits = f.logits, c.bias = r.bias;
    c.idx = r.idx, c.weights = r.weights, c.E = r.E, c.d = a.gate.K, c.f = a.gate.N, c.T = (int)a.T, c.k = r.k;
    c.gx = (a.gate.nb + 1) / 2, c.dx = a.down.nb, c.ldh = (int)f.ldh, c.patience = f.patience;
    c.groups = r.groups, c.keep = r.keep, c.per_group = r.E / r.groups, c.log_lanes = route_log_lanes(r.groups);
    c.flags = (r.sigmoid ? kFewSigmoid : 0) | (r.renorm ? kFewRenorm : 0) | (r.group_top == 2 ? kFewTopTwo : 0) |
              (route_own(r.E, r.groups) <= 1 ? kFewOne : 0);
    const int parts = a.dtype == kF32 ? 3 : 2;
    const size_t up = q4_row_lds(a.gate.ku, a.dtype == kF32 ? 3 : 1), down = q4_row_lds((int64_t)r.k * a.down.ku, parts);
    const size_t lds = up > down ? up : down;
    if (a.dtype == kF16) return run<kXF16, kXF32x2, 2, kF16>(c, a, lds, s);
    if (a.dtype == kBF16) return run<kXBF16, kXF32x2, 2, kBF16>(c, a, lds, s);
    return run<kXF32x3, kXF32x3, 3, kF32>(c, a, lds, s);
}

}  // namespace tq2
