// Experts' gated products over 4-bit weights: for each token t and slot j with
// expert e = idx[t][j],
//   y[t] = sum_j weight[t][j] * down_e( silu(gate_e x_t) * (up_e x_t) ),
// slots whose idx is outside 0 .. E-1 dropped.  Four launches: the plan (slots
// sorted by expert, and the list of row tiles), the gate and up products with
// silu(g) u in their epilogue, the down product times the slot's weight, and the
// sum of each token's slots in slot order.
#include "q4_skinny.h"

namespace tq2 {

namespace {

constexpr int kMaxExperts = 1024;

// One workgroup.  Counts and places come from LDS atomics: the order of slots
// within an expert may differ from call to call, but a slot's products do not
// depend on its place, and the sum over slots goes by slot, so results are the
// same bits.
__global__ __launch_bounds__(1024) void moe_plan_kernel(const int32_t *idx, int slots, int E, int tile_rows,
                                                        int32_t *order, int4 *tiles, int32_t *ntiles) {
    __shared__ int cnt[kMaxExperts], base[kMaxExperts], tbase[kMaxExperts];
    const int tid = threadIdx.x;
    for (int e = tid; e < E; e += 1024) cnt[e] = 0;
    __syncthreads();
    for (int s = tid; s < slots; s += 1024) {
        const int e = idx[s];
        if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    // inclusive scans of the slots and of the tiles, in place
    if (tid < E) base[tid] = cnt[tid], tbase[tid] = (cnt[tid] + tile_rows - 1) / tile_rows;
    __syncthreads();
    for (int o = 1; o < E; o <<= 1) {
        int a = 0, b = 0;
        if (tid < E && tid >= o) a = base[tid - o], b = tbase[tid - o];
        __syncthreads();
        if (tid < E) base[tid] += a, tbase[tid] += b;
        __syncthreads();
    }
    if (tid == E - 1) *ntiles = tbase[tid];
    int first = 0, c = 0;
    if (tid < E) {
        c = cnt[tid];
        first = base[tid] - c;
        int t = tbase[tid] - (c + tile_rows - 1) / tile_rows;
        for (int r = 0; r < c; r += tile_rows, ++t)
            tiles[t] = int4{tid, first + r, c - r < tile_rows ? c - r : tile_rows, 0};
    }
    __syncthreads();
    if (tid < E) cnt[tid] = first;  // the next free place
    __syncthreads();
    for (int s = tid; s < slots; s += 1024) {
        const int e = idx[s];
        if (e >= 0 && e < E) order[atomicAdd(&cnt[e], 1)] = s;
    }
}

template <int DT>
__global__ __launch_bounds__(256) void moe_sum_kernel(const float *part, const int32_t *idx, void *y, int64_t T, int k,
                                                      int E, int d) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= T * d) return;
    const int64_t t = i / d;
    const int n = (int)(i % d);
    f4 v = {};
    for (int j = 0; j < k; ++j) {
        const int e = idx[t * k + j];
        if (e >= 0 && e < E) v += *reinterpret_cast<const f4 *>(part + (t * k + j) * d + n);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) store_from_float<DT>(y, i + q, v[q]);
}

template <int XT, int G, int MODE>
hipError_t product_rb(const MoePlan &p, const Q4Args &a, hipStream_t s) {
    return p.tile_rows == 16 ? run_q4_skinny<XT, G, 1, 2, MODE>(a, p.max_tiles, s)
                             : run_q4_skinny<XT, G, 2, 2, MODE>(a, p.max_tiles, s);
}

template <int XT, int MODE>
hipError_t product(const MoePlan &p, const Q4Args &a, hipStream_t s) {
    if (a.w.G == 32) return product_rb<XT, 32, MODE>(p, a, s);
    if (a.w.G == 64) return product_rb<XT, 64, MODE>(p, a, s);
    return product_rb<XT, 128, MODE>(p, a, s);
}

}  // namespace

MoePlan moe_plan(int64_t T, int64_t k, int64_t E, int64_t d, int64_t f, int dtype) {
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    MoePlan p{};
    (void)dtype;
    p.slots = T * k;
    p.tile_rows = p.slots <= 16 * E ? 16 : 32;
    p.max_tiles = p.slots / p.tile_rows + (E < p.slots ? E : p.slots);
    p.off_order = 256;  // the first 256 bytes hold the number of tiles
    p.off_tiles = p.off_order + up((size_t)p.slots * 4);
    p.off_h = p.off_tiles + up((size_t)p.max_tiles * 16);
    p.off_part = p.off_h + up((size_t)p.slots * f * 4);
    p.total = p.off_part + up((size_t)p.slots * d * 4);
    return p;
}

hipError_t launch_q4_moe(const MoePlan &p, const void *x, const int32_t *idx, const float *weights, const Q4View &gate,
                         const Q4View &up, const Q4View &down, void *y, int64_t T, int64_t k, int dtype, void *ws,
                         hipStream_t s) {
    char *b = static_cast<char *>(ws);
    int32_t *ntiles = reinterpret_cast<int32_t *>(b), *order = reinterpret_cast<int32_t *>(b + p.off_order);
    int4 *tiles = reinterpret_cast<int4 *>(b + p.off_tiles);
    float *h = reinterpret_cast<float *>(b + p.off_h), *part = reinterpret_cast<float *>(b + p.off_part);
    moe_plan_kernel<<<dim3(1), dim3(1024), 0, s>>>(idx, (int)p.slots, gate.E, (int)p.tile_rows, order, tiles, ntiles);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    Q4Args g{};
    g.w = gate, g.w2 = up, g.x = x, g.y = h, g.topk = (int)k, g.order = order, g.tiles = tiles, g.ntiles = ntiles;
    g.weights = weights;
    Q4Args d = g;
    d.w = down, d.x = h, d.y = part;
    if (dtype == kF16) e = product<kXF16, kGateUp>(p, g, s);
    else if (dtype == kBF16) e = product<kXBF16, kGateUp>(p, g, s);
    else e = product<kXF32x3, kGateUp>(p, g, s);
    if (e != hipSuccess) return e;
    // h for a 16-bit result is taken in 16 bits (two bfloat16 parts, relative error 2^-17)
    e = dtype == kF32 ? product<kXF32x3, kDown>(p, d, s) : product<kXF32x2, kDown>(p, d, s);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((T * down.N / 4 + 255) / 256));
    if (dtype == kF16) moe_sum_kernel<kF16><<<grid, dim3(256), 0, s>>>(part, idx, y, T, (int)k, gate.E, down.N);
    else if (dtype == kBF16) moe_sum_kernel<kBF16><<<grid, dim3(256), 0, s>>>(part, idx, y, T, (int)k, gate.E, down.N);
    else moe_sum_kernel<kF32><<<grid, dim3(256), 0, s>>>(part, idx, y, T, (int)k, gate.E, down.N);
    return hipGetLastError();
}

}  // namespace tq2
