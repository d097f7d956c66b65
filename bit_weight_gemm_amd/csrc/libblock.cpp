// C ABI of a block's parts around 4-bit weights: argument checks and launches.  Declarations and the contract live in
// include/libtq2_block.h.
#include <hip/hip_runtime.h>

#include <atomic>

#include "../../include/libtq2_block.h"
#include "block_norm.h"
#include "checks.h"
#include "internal.h"
#include "moe_layer.h"
#include "q4_epilogue.h"

using namespace tq2::check;

namespace {

// A tensor of a call: where it is, its bytes, the alignment of its address.
struct Tensor {
    const void *at;
    size_t bytes;
    uintptr_t align;
};

bool misaligned(std::initializer_list<Tensor> all) {
    for (const Tensor &t : all)
        if (!aligned(t.at, t.align)) return true;
    return false;
}

// Whether some output overlaps another output or an input (absent ones are null and overlap nothing).
bool clash(std::initializer_list<Tensor> outs, std::initializer_list<Tensor> ins) {
    auto meet = [](const Tensor &a, const Tensor &b) { return a.at && b.at && overlap(a.at, a.bytes, b.at, b.bytes); };
    for (const Tensor &o : outs) {
        for (const Tensor &i : ins)
            if (meet(o, i)) return true;
        for (const Tensor &q : outs)
            if (&q != &o && meet(o, q)) return true;
    }
    return false;
}

bool clash_workspace(const void *ws, size_t need, std::initializer_list<Tensor> a, std::initializer_list<Tensor> b) {
    for (auto list : {a, b})
        for (const Tensor &t : list)
            if (t.at && overlap(ws, need, t.at, t.bytes)) return true;
    return false;
}

bool side_type(int type, int dtype) { return type == Q4_F32 || type == dtype; }

constexpr int64_t kNormColumns = 16384;

// Some tens of milliseconds, and no call may wait longer.
constexpr int kMostPatience = 1 << 16;
std::atomic<int> g_patience{kMostPatience};

bool norm_sizes(int64_t M, int64_t N, int64_t R, int dtype) {
    return M >= 0 && M <= kMaxRows && N >= 1 && N <= kNormColumns && R >= 1 && (M == 0 || (R <= M && M % R == 0)) && known(dtype);
}

}  // namespace

extern "C" {

int q4_linear(const q4_weight *w, const void *x, const void *bias, int bias_dtype, int activation, const void *residual,
              void *y, int64_t M, int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (!weight_ok(w) || w->E != 1 || !known(dtype) || M < 0 || M > kMaxRows) return TQ2_EINVAL;
    if (activation < Q4_ACT_NONE || activation > Q4_ACT_SILU || (bias && !side_type(bias_dtype, dtype))) return TQ2_EINVAL;
    if (M == 0) return tq2::current_device(nullptr);
    const size_t s = size_of(dtype), ybytes = (size_t)M * w->N * s, need = q4_gemm_workspace_size(w, M, dtype);
    const Tensor out{y, ybytes, 16}, in{x, (size_t)M * w->K * s, 16}, packed{w->data, bytes(w), 256};
    const Tensor add{residual, ybytes, 16}, vec{bias, (size_t)w->N * size_of(bias_dtype), size_of(bias_dtype)};
    if (!x || !y || misaligned({out, in, add}) || (bias && misaligned({vec}))) return TQ2_EINVAL;
    if (clash({out}, {in, packed, vec}) || (residual != y && clash({out}, {add}))) return TQ2_EINVAL;
    if (need && (workspace_bad(workspace, workspace_bytes, need, {}) ||
                 clash_workspace(workspace, need, {out, in, packed}, {add, vec})))
        return TQ2_EINVAL;
    const int st = tq2::current_device(nullptr);
    if (st) return st;
    tq2::Q4Epilogue epi{};
    epi.bias = bias, epi.residual = residual, epi.bias_f32 = bias_dtype == Q4_F32, epi.act = activation;
    return tq2::status_of(tq2::launch_q4_gemm(view(w), x, y, M, dtype, workspace, &epi, static_cast<hipStream_t>(stream)));
}

size_t moe_layer_workspace_size(int64_t T, int64_t k, int64_t E, int64_t d, int64_t f, int dtype, int with_norm) {
    if (q4_moe_workspace_size(T, k, E, d, f, dtype) == 0 || k > E) return 0;
    return tq2::layer_plan(T, k, E, 1, d, f, dtype, with_norm != 0, false).total;
}

int moe_layer(const moe_layer_call *c, void *workspace, size_t workspace_bytes, void *stream) {
    if (!c || !weight_ok(c->gate) || !weight_ok(c->up) || !weight_ok(c->down) || !known(c->dtype)) return TQ2_EINVAL;
    const q4_weight *gate = c->gate, *up = c->up, *down = c->down;
    const int64_t E = gate->E, f = gate->N, d = gate->K, T = c->T, k = c->k;
    if (up->E != E || up->N != f || up->K != d || up->G != gate->G || up->zeros != gate->zeros || down->E != E ||
        down->N != d || down->K != f)
        return TQ2_EINVAL;
    if (!side_type(c->router_dtype, c->dtype) || (c->norm && (!side_type(c->norm_dtype, c->dtype) || d > kNormColumns)))
        return TQ2_EINVAL;
    if (c->groups < 1 || c->groups > 64 || E % c->groups || c->keep < 1 || c->keep > c->groups || c->group_top < 1 ||
        c->group_top > 2 || (c->score != MOE_SOFTMAX && c->score != MOE_SIGMOID))
        return TQ2_EINVAL;
    const size_t need = moe_layer_workspace_size(T, k, E, d, f, c->dtype, c->norm != nullptr);
    if (need == 0) return TQ2_EINVAL;
    if (T == 0) return tq2::current_device(nullptr);
    const size_t rows = (size_t)T * d * size_of(c->dtype), slots = (size_t)T * k * 4;
    const Tensor y{c->y, rows, 16}, idx{c->idx, slots, 4}, weights{c->weights, slots, 4};
    const Tensor x{c->x, rows, 16}, residual{c->residual, rows, 16};
    const Tensor router{c->router, (size_t)E * d * size_of(c->router_dtype), 16};
    const Tensor norm{c->norm, (size_t)d * size_of(c->norm_dtype), size_of(c->norm_dtype)}, bias{c->bias, (size_t)E * 4, 4};
    const Tensor wg{gate->data, bytes(gate), 256}, wu{up->data, bytes(up), 256}, wd{down->data, bytes(down), 256};
    if (!c->x || !c->router || !c->y || !c->idx || !c->weights || misaligned({y, idx, weights, x, residual, router, bias}) ||
        (c->norm && misaligned({norm})))
        return TQ2_EINVAL;
    if (clash({y, idx, weights}, {x, router, norm, bias, wg, wu, wd}) || clash({idx, weights}, {residual}) ||
        (c->residual != c->y && clash({y}, {residual})))
        return TQ2_EINVAL;
    if (workspace_bad(workspace, workspace_bytes, need, {}) ||
        clash_workspace(workspace, need, {y, idx, weights, residual}, {x, router, norm, bias, wg, wu, wd}))
        return TQ2_EINVAL;
    const int st = tq2::current_device(nullptr);
    if (st) return st;
    tq2::LayerArgs a{};
    a.x = c->x, a.norm = c->norm, a.router = c->router, a.residual = c->residual, a.y = c->y, a.T = T, a.dtype = c->dtype;
    a.wide_norm = c->norm_dtype == Q4_F32, a.wide_router = c->router_dtype == Q4_F32, a.eps = c->eps;
    a.gate = view(gate), a.up = view(up), a.down = view(down);
    a.route.bias = c->bias, a.route.idx = c->idx, a.route.weights = c->weights, a.route.T = T;
    a.route.E = (int)E, a.route.k = (int)k, a.route.groups = (int)c->groups, a.route.keep = (int)c->keep;
    a.route.group_top = (int)c->group_top, a.route.sigmoid = c->score == MOE_SIGMOID, a.route.renorm = c->renorm != 0;
    const bool coarse = gate->G == tq2::kFewGroup && down->G == tq2::kFewGroup;
    const tq2::LayerPlan p = tq2::layer_plan(T, k, E, c->groups, d, f, c->dtype, c->norm != nullptr, coarse);
    return tq2::status_of(tq2::launch_moe_layer(p, a, workspace, g_patience, static_cast<hipStream_t>(stream)));
}

int moe_layer_set_patience(int tries) {
    if (tries < 0 || tries > kMostPatience) return TQ2_EINVAL;
    return g_patience.exchange(tries);
}

int block_norm(const block_norm_call *c, void *stream) {
    if (!c || !norm_sizes(c->M, c->N, c->R, c->dtype) || !side_type(c->weights_dtype, c->dtype)) return TQ2_EINVAL;
    if (c->M == 0) return tq2::current_device(nullptr);
    if ((!c->b && (c->post || c->gate || c->y)) || (!c->post && c->post_bias) || (!c->pre && (c->pre_bias || c->n)))
        return TQ2_EINVAL;
    if ((c->pre && !c->n) || (!c->y && !c->n) || (!c->gate && c->R != 1)) return TQ2_EINVAL;
    const size_t s = size_of(c->dtype), ws = size_of(c->weights_dtype), rows = (size_t)c->M * c->N * s, vec = (size_t)c->N * ws;
    const Tensor x{c->x, rows, s}, b{c->b, rows, s}, y{c->y, rows, s}, n{c->n, rows, s}, gate{c->gate, vec * c->R, ws};
    const Tensor post{c->post, vec, ws}, post_bias{c->post_bias, vec, ws}, pre{c->pre, vec, ws}, pre_bias{c->pre_bias, vec, ws};
    if (!c->x || misaligned({x, b, y, n, gate, post, post_bias, pre, pre_bias})) return TQ2_EINVAL;
    if (clash({y, n}, {x, b, gate, post, post_bias, pre, pre_bias})) return TQ2_EINVAL;
    const int st = tq2::current_device(nullptr);
    if (st) return st;
    tq2::BlockNormArgs a{};
    a.x = c->x, a.b = c->b, a.post = c->post, a.post_bias = c->post_bias, a.gate = c->gate, a.pre = c->pre;
    a.pre_bias = c->pre_bias, a.y = c->y, a.n = c->n, a.M = c->M, a.gate_rows = c->M / c->R, a.N = (int)c->N;
    a.layer = c->layer != 0, a.scale = c->scale, a.eps = c->eps;
    return tq2::status_of(tq2::launch_block_norm(a, c->dtype, c->weights_dtype == Q4_F32, static_cast<hipStream_t>(stream)));
}

size_t block_norm_backward_workspace_size(int64_t M, int64_t N, int64_t R, int dtype) {
    return norm_sizes(M, N, R, dtype) ? tq2::block_norm_backward_workspace(M, N, R, dtype) : 0;
}

int block_norm_backward(const block_norm_backward_call *c, void *workspace, size_t workspace_bytes, void *stream) {
    if (!c || !norm_sizes(c->M, c->N, c->R, c->dtype) || !side_type(c->weights_dtype, c->dtype)) return TQ2_EINVAL;
    if ((!c->post && (c->post_bias || c->dpost || c->dpost_bias)) || (!c->gate && (c->dgate || c->R != 1)) ||
        (!c->pre && (c->pre_bias || c->dpre || c->dpre_bias)))
        return TQ2_EINVAL;
    // (a call without rows has no row tensors, and zeros for sums)
    if (c->M && ((!c->b && (c->post || c->gate || c->db)) || (c->pre && (!c->dn || !c->y)) || (!c->pre && (c->dn || c->y)) ||
                 (!c->dy && !c->dn)))
        return TQ2_EINVAL;
    const size_t s = size_of(c->dtype), ws = size_of(c->weights_dtype), rows = (size_t)c->M * c->N * s, vec = (size_t)c->N * ws;
    const size_t need = tq2::block_norm_backward_workspace(c->M, c->N, c->R, c->dtype), sums = (size_t)c->N * 4;
    const Tensor dy{c->dy, rows, s}, dn{c->dn, rows, s}, y{c->y, rows, s}, b{c->b, rows, s}, gate{c->gate, vec * c->R, ws};
    const Tensor post{c->post, vec, ws}, post_bias{c->post_bias, vec, ws}, pre{c->pre, vec, ws}, pre_bias{c->pre_bias, vec, ws};
    const Tensor dx{c->dx, rows, s}, db{c->db, rows, s}, dgate{c->dgate, sums * c->R, 4}, dpost{c->dpost, sums, 4};
    const Tensor dpost_bias{c->dpost_bias, sums, 4}, dpre{c->dpre, sums, 4}, dpre_bias{c->dpre_bias, sums, 4};
    if (misaligned({dy, dn, y, b, gate, post, post_bias, pre, pre_bias}) ||
        misaligned({dx, db, dgate, dpost, dpost_bias, dpre, dpre_bias}))
        return TQ2_EINVAL;
    if (clash({dx, db, dgate, dpost, dpost_bias, dpre, dpre_bias}, {dy, dn, y, b, gate, post, post_bias, pre, pre_bias}))
        return TQ2_EINVAL;
    if (need && (workspace_bad(workspace, workspace_bytes, need, {}) ||
                 clash_workspace(workspace, need, {dy, dn, y, b, gate, post, post_bias, pre, pre_bias},
                                 {dx, db, dgate, dpost, dpost_bias, dpre, dpre_bias})))
        return TQ2_EINVAL;
    const int st = tq2::current_device(nullptr);
    if (st) return st;
    tq2::BlockNormBackwardArgs a{};
    a.dy = c->dy, a.dn = c->dn, a.y = c->y, a.b = c->b, a.post = c->post, a.post_bias = c->post_bias, a.gate = c->gate;
    a.pre = c->pre, a.pre_bias = c->pre_bias, a.dx = c->dx, a.db = c->db, a.dpost = c->dpost, a.dpost_bias = c->dpost_bias;
    a.dgate = c->dgate, a.dpre = c->dpre, a.dpre_bias = c->dpre_bias, a.M = c->M;
    a.gate_rows = c->M ? c->M / c->R : c->R;  // (without rows: for dgate's size)
    a.N = (int)c->N, a.layer = c->layer != 0, a.scale = c->scale, a.eps = c->eps;
    return tq2::status_of(tq2::launch_block_norm_backward(a, c->dtype, c->weights_dtype == Q4_F32, workspace,
                                                          static_cast<hipStream_t>(stream)));
}

}  // extern "C"
