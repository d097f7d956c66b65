// C ABI of the 4-bit weights and the mixture-of-experts operators: argument checks
// and launches.  Declarations and the contract live in include/libtq2_moe.h.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "../../include/libtq2_moe.h"
#include "internal.h"
#include "q4.h"

namespace {

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

size_t size_of(int dtype) { return dtype == Q4_F32 ? 4 : 2; }

bool known(int dtype) { return dtype == Q4_F32 || dtype == Q4_F16 || dtype == Q4_BF16; }

bool weight_ok(const q4_weight *w) {
    return w && w->data && aligned(w->data, 256) && (w->zeros == 0 || w->zeros == 1) &&
           q4_packed_size(w->E, w->N, w->K, w->G, w->zeros) != 0;
}

tq2::Q4View view(const q4_weight *w) { return tq2::q4_view(w->data, w->E, w->N, w->K, w->G, w->zeros != 0); }

size_t bytes(const q4_weight *w) { return q4_packed_size(w->E, w->N, w->K, w->G, w->zeros); }

struct Range {
    const void *at;
    size_t bytes;
};

// A caller's workspace: large enough, 256-byte aligned, clear of the call's other arguments.
bool workspace_bad(const void *ws, size_t ws_bytes, size_t need, std::initializer_list<Range> others) {
    if (!ws || ws_bytes < need || !aligned(ws, 256)) return true;
    for (const Range &r : others)
        if (overlap(ws, need, r.at, r.bytes)) return true;
    return false;
}

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;

}  // namespace

extern "C" {

size_t q4_packed_size(int64_t E, int64_t N, int64_t K, int64_t G, int zeros) {
    if (E < 1 || E > 1024 || N < 1 || N > ((int64_t)1 << 24) || (G != 32 && G != 64 && G != 128)) return 0;
    if (K < G || K % G || K > ((int64_t)1 << 20)) return 0;
    return tq2::q4_layout(E, N, K, G, zeros != 0).total;
}

int q4_pack(const q4_weight *w, const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, void *stream) {
    if (!weight_ok(w) || !codes || !scales || (zeros != nullptr) != (w->zeros == 1)) return TQ2_EINVAL;
    if (!aligned(codes, 4) || !aligned(scales, 2)) return TQ2_EINVAL;
    const size_t n = (size_t)w->E * w->N, groups = n * (w->K / w->G);
    if (overlap(w->data, bytes(w), codes, n * w->K / 2) || overlap(w->data, bytes(w), scales, groups * 2) ||
        overlap(w->data, bytes(w), zeros, zeros ? groups : 0))
        return TQ2_EINVAL;
    const int st = tq2::current_device(nullptr);
    if (st) return st;
    return tq2::status_of(tq2::launch_q4_pack(codes, scales, zeros, view(w), static_cast<hipStream_t>(stream)));
}

int q4_dequant(const q4_weight *w, float *w_out, void *stream) {
    if (!weight_ok(w) || !w_out || !aligned(w_out, 4)) return TQ2_EINVAL;
    if (overlap(w->data, bytes(w), w_out, (size_t)w->E * w->N * w->K * 4)) return TQ2_EINVAL;
    const int st = tq2::current_device(nullptr);
    if (st) return st;
    return tq2::status_of(tq2::launch_q4_dequant(view(w), w_out, static_cast<hipStream_t>(stream)));
}

size_t q4_gemm_workspace_size(const q4_weight *w, int64_t M, int dtype) {
    if (!w || q4_packed_size(w->E, w->N, w->K, w->G, w->zeros) == 0 || M < 0 || M > kMaxRows || !known(dtype)) return 0;
    return tq2::q4_gemm_workspace(w->N, w->K, w->G, M, dtype);
}

int q4_gemm(const q4_weight *w, const void *x, void *y, int64_t M, int dtype, void *workspace, size_t workspace_bytes,
            void *stream) {
    if (!weight_ok(w) || w->E != 1 || !known(dtype) || M < 0 || M > kMaxRows) return TQ2_EINVAL;
    if (M == 0) return tq2::current_device(nullptr);
    if (!x || !y || !aligned(x, 16) || !aligned(y, 16)) return TQ2_EINVAL;
    const size_t ybytes = (size_t)M * w->N * size_of(dtype), need = q4_gemm_workspace_size(w, M, dtype);
    const size_t xbytes = (size_t)M * w->K * size_of(dtype);
    if (overlap(y, ybytes, x, xbytes) || overlap(y, ybytes, w->data, bytes(w))) return TQ2_EINVAL;
    if (need && workspace_bad(workspace, workspace_bytes, need, {{y, ybytes}, {x, xbytes}, {w->data, bytes(w)}}))
        return TQ2_EINVAL;
    const int st = tq2::current_device(nullptr);
    if (st) return st;
    return tq2::status_of(tq2::launch_q4_gemm(view(w), x, y, M, dtype, workspace, static_cast<hipStream_t>(stream)));
}

int moe_route(const void *logits, const float *bias, int32_t *idx, float *weights, int64_t T, int64_t E, int64_t k,
              int64_t groups, int64_t keep, int64_t group_top, int score, int renorm, int dtype, void *stream) {
    if (T < 0 || T > kMaxRows || E < 1 || E > 1024 || k < 1 || k > 64 || k > E || !known(dtype)) return TQ2_EINVAL;
    if (groups < 1 || groups > 64 || E % groups || keep < 1 || keep > groups || group_top < 1 || group_top > 2)
        return TQ2_EINVAL;
    if (score != MOE_SOFTMAX && score != MOE_SIGMOID) return TQ2_EINVAL;
    if (T == 0) return tq2::current_device(nullptr);
    if (!logits || !idx || !weights || !aligned(logits, size_of(dtype)) || !aligned(bias, 4) || !aligned(idx, 4) ||
        !aligned(weights, 4))
        return TQ2_EINVAL;
    const size_t in = (size_t)T * E * size_of(dtype), out = (size_t)T * k * 4;
    if (overlap(idx, out, weights, out) || overlap(idx, out, logits, in) || overlap(weights, out, logits, in) ||
        (bias && (overlap(idx, out, bias, E * 4) || overlap(weights, out, bias, E * 4))))
        return TQ2_EINVAL;
    const int st = tq2::current_device(nullptr);
    if (st) return st;
    tq2::RouteArgs a{};
    a.logits = logits, a.bias = bias, a.idx = idx, a.weights = weights, a.T = T;
    a.E = (int)E, a.k = (int)k, a.groups = (int)groups, a.keep = (int)keep, a.group_top = (int)group_top;
    a.dtype = dtype, a.sigmoid = score == MOE_SIGMOID, a.renorm = renorm != 0;
    return tq2::status_of(tq2::launch_moe_route(a, static_cast<hipStream_t>(stream)));
}

int moe_route_backward(const void *logits, const int32_t *idx, const float *dw, void *dlogits, int64_t T, int64_t E,
                       int64_t k, int score, int renorm, int dtype, void *stream) {
    if (T < 0 || T > kMaxRows || E < 1 || E > 1024 || k < 1 || k > 64 || !known(dtype)) return TQ2_EINVAL;
    if (score != MOE_SOFTMAX && score != MOE_SIGMOID) return TQ2_EINVAL;
    if (T == 0) return tq2::current_device(nullptr);
    if (!logits || !idx || !dw || !dlogits || !aligned(logits, size_of(dtype)) || !aligned(dlogits, size_of(dtype)) ||
        !aligned(idx, 4) || !aligned(dw, 4))
        return TQ2_EINVAL;
    const size_t n = (size_t)T * E * size_of(dtype), m = (size_t)T * k * 4;
    if (overlap(dlogits, n, logits, n) || overlap(dlogits, n, idx, m) || overlap(dlogits, n, dw, m)) return TQ2_EINVAL;
    const int st = tq2::current_device(nullptr);
    if (st) return st;
    return tq2::status_of(tq2::launch_moe_route_backward(logits, idx, dw, dlogits, T, (int)E, (int)k, dtype,
                                                         score == MOE_SIGMOID, renorm != 0,
                                                         static_cast<hipStream_t>(stream)));
}

size_t q4_moe_workspace_size(int64_t T, int64_t k, int64_t E, int64_t d, int64_t f, int dtype) {
    if (T < 0 || k < 1 || k > 64 || T >= ((int64_t)1 << 24) / k || E < 1 || E > 1024 || !known(dtype)) return 0;
    if (q4_packed_size(E, f, d, 32, 0) == 0 || q4_packed_size(E, d, f, 32, 0) == 0) return 0;
    return tq2::moe_plan(T, k, E, d, f, dtype).total;
}

int q4_moe(const void *x, const int32_t *idx, const float *weights, const q4_weight *gate, const q4_weight *up,
           const q4_weight *down, void *y, int64_t T, int64_t k, int dtype, void *workspace, size_t workspace_bytes,
           void *stream) {
    if (!weight_ok(gate) || !weight_ok(up) || !weight_ok(down) || !known(dtype)) return TQ2_EINVAL;
    const int64_t E = gate->E, f = gate->N, d = gate->K;
    if (up->E != E || up->N != f || up->K != d || up->G != gate->G || up->zeros != gate->zeros || down->E != E ||
        down->N != d || down->K != f)
        return TQ2_EINVAL;
    const size_t need = q4_moe_workspace_size(T, k, E, d, f, dtype);
    if (need == 0) return TQ2_EINVAL;
    if (T == 0) return tq2::current_device(nullptr);
    if (!x || !idx || !weights || !y || !aligned(x, 16) || !aligned(y, 16) || !aligned(idx, 4) || !aligned(weights, 4))
        return TQ2_EINVAL;
    const size_t n = (size_t)T * d * size_of(dtype), m = (size_t)T * k * 4;
    if (overlap(y, n, x, n) || overlap(y, n, idx, m) || overlap(y, n, weights, m) || overlap(y, n, gate->data, bytes(gate)) ||
        overlap(y, n, up->data, bytes(up)) || overlap(y, n, down->data, bytes(down)))
        return TQ2_EINVAL;
    if (workspace_bad(workspace, workspace_bytes, need,
                      {{y, n}, {x, n}, {idx, m}, {weights, m}, {gate->data, bytes(gate)}, {up->data, bytes(up)},
                       {down->data, bytes(down)}}))
        return TQ2_EINVAL;
    const int st = tq2::current_device(nullptr);
    if (st) return st;
    const tq2::MoePlan p = tq2::moe_plan(T, k, E, d, f, dtype);
    return tq2::status_of(tq2::launch_q4_moe(p, x, idx, weights, view(gate), view(up), view(down), y, T, k, dtype,
                                             workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
