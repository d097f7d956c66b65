// Experts' gated products over 4-bit weights: for each token t and slot j with
// expert e = idx[t][j],
//   y[t] = sum_j weight[t][j] * down_e( silu(gate_e x_t) * (up_e x_t) ),
// slots whose idx is outside 0 .. E-1 dropped.  With many slots four launches: the plan
// (slots sorted by expert, and the list of row tiles; beside it x as f16 planes), the
// gate and up products with silu(g) u in their epilogue, the down product times the
// slot's weight, and the sum of each token's slots in slot order.  With fewer, three
// without the plan, with a few two; moe_plan says when.
#include "q4_group.h"
#include "q4_prep.h"
#include "q4_row.h"

namespace tq2 {

namespace {

constexpr int kMaxExperts = 1024;

// One workgroup (16384 slots: 13 us beside the planes of 2048 rows, alone 11.6, bound by its one compute unit's atomics and the two passes' latency).
// Counts and places come from LDS atomics: the order of slots
// within an expert may differ from call to call, but a slot's products do not
// depend on its place, and the sum over slots goes by slot, so results are the
// same bits.
// The other workgroups bring x's rows to f16 planes meanwhile (sixteen rows each; none if x.rows is 0).
template <int DT, int P>
__global__ __launch_bounds__(1024) void moe_plan_kernel(const int32_t *idx, int slots, int E, int tile_rows,
                                                        int32_t *order, int4 *tiles, int32_t *ntiles, Q4Prep x) {
    if (blockIdx.x > 0) {
        const int64_t row = (int64_t)(blockIdx.x - 1) * 16 + (threadIdx.x >> 6);
        if (row < x.rows) q4_prep_row<DT, P>(x, row);
        return;
    }
    __shared__ int cnt[kMaxExperts], base[kMaxExperts], tbase[kMaxExperts];
    const int tid = threadIdx.x;
    for (int e = tid; e < E; e += 1024) cnt[e] = 0;
    __syncthreads();
    // sixteen slots of a thread at a time: their loads, then their atomics, wait together
    // (16384 slots: 16 us one by one)
    constexpr int kBatch = 16;
    for (int s0 = tid; s0 < slots; s0 += 1024 * kBatch) {
        int e[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) e[i] = s0 + 1024 * i < slots ? idx[s0 + 1024 * i] : -1;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (e[i] >= 0 && e[i] < E) atomicAdd(&cnt[e[i]], 1);
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
    for (int s0 = tid; s0 < slots; s0 += 1024 * kBatch) {
        int e[kBatch], at[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) e[i] = s0 + 1024 * i < slots ? idx[s0 + 1024 * i] : -1;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) at[i] = e[i] >= 0 && e[i] < E ? atomicAdd(&cnt[e[i]], 1) : -1;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (at[i] >= 0) order[at[i]] = s0 + 1024 * i;
    }
}

// The slots' parts of each token, in slot order: 2048 tokens of 8 slots, 2048 wide, 22 us (142 MB, 6.4 TB/s:
// in part from the last-level cache).
template <int DT>
__global__ __launch_bounds__(256) void moe_sum_kernel(const float *part, const int32_t *idx, void *y, int64_t T, int k,
                                                      int E, int d) {
    const int64_t step = (int64_t)gridDim.x * 1024;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < T * d; i += step) {
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
}

template <int XT, int MODE>
hipError_t product(const MoePlan &p, const Q4Args &a, hipStream_t s) {
    if (a.w.G == 32) return run_q4_skinny<XT, 32, 1, 2, MODE>(a, p.max_tiles, s);
    if (a.w.G == 64) return run_q4_skinny<XT, 64, 1, 2, MODE>(a, p.max_tiles, s);
    return run_q4_skinny<XT, 128, 1, 2, MODE>(a, p.max_tiles, s);
}

// Two column blocks of each product to a workgroup (one token 13.8 us, with one 14.5; 64 slots 45 and 52); two
// units of codes in flight in either launch.
template <int XT, int PH>
hipError_t row_gate_up(const Q4RowArgs &a, int64_t slots, hipStream_t s) {
    if (a.w.G == 32) return run_q4_row<XT, 32, 4, 8, 2, kRowGateUp, PH, kF32>(a, slots, s);
    if (a.w.G == 64) return run_q4_row<XT, 64, 4, 8, 2, kRowGateUp, PH, kF32>(a, slots, s);
    return run_q4_row<XT, 128, 4, 8, 2, kRowGateUp, PH, kF32>(a, slots, s);
}

template <int XT, int DT>
hipError_t row_down_sum(const Q4RowArgs &a, int64_t T, hipStream_t s) {
    if (a.w.G == 32) return run_q4_row<XT, 32, 1, 16, 2, kRowDownSum, 1, DT>(a, T, s);
    if (a.w.G == 64) return run_q4_row<XT, 64, 1, 16, 2, kRowDownSum, 1, DT>(a, T, s);
    return run_q4_row<XT, 128, 1, 16, 2, kRowDownSum, 1, DT>(a, T, s);
}

// A few slots: two launches, every slot with its own expert's weights; h in two
// bfloat16 parts (relative error 2^-17) for 16-bit types, in three, which are exact, for f32.
hipError_t direct(const MoePlan &p, const void *x, const int32_t *idx, const float *weights, const Q4View &gate,
                  const Q4View &up, const Q4View &down, void *y, int64_t T, int64_t k, int dtype, char *b, hipStream_t s) {
    Q4RowArgs g{};
    g.w = gate, g.w2 = up, g.x = x, g.y = b + p.off_h, g.topk = (int)k, g.weights = weights, g.idx = idx, g.ldh = p.ldh;
    hipError_t e;
    if (dtype == kF16) e = row_gate_up<kXF16, 2>(g, p.slots, s);
    else if (dtype == kBF16) e = row_gate_up<kXBF16, 2>(g, p.slots, s);
    else e = row_gate_up<kXF32x3, 3>(g, p.slots, s);
    if (e != hipSuccess) return e;
    Q4RowArgs d = g;
    d.w = down, d.x = g.y, d.y = y;
    if (dtype == kF16) return row_down_sum<kXF32x2, kF16>(d, T, s);
    if (dtype == kBF16) return row_down_sum<kXF32x2, kBF16>(d, T, s);
    return row_down_sum<kXF32x3, kF32>(d, T, s);
}

template <int DT>
void launch_sum(const float *part, const int32_t *idx, void *y, int64_t T, int64_t k, int E, int d, hipStream_t s) {
    const int64_t blocks = (T * d / 4 + 255) / 256, most = (int64_t)1 << 20;
    moe_sum_kernel<DT><<<dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, s>>>(part, idx, y, T, (int)k, E, d);
}

hipError_t sum(const float *part, const int32_t *idx, void *y, int64_t T, int64_t k, int E, int d, int dtype, hipStream_t s) {
    if (dtype == kF16) launch_sum<kF16>(part, idx, y, T, k, E, d, s);
    else if (dtype == kBF16) launch_sum<kBF16>(part, idx, y, T, k, E, d, s);
    else launch_sum<kF32>(part, idx, y, T, k, E, d, s);
    return hipGetLastError();
}

// A few rows per expert: every expert's workgroups find their slots, no plan.  As in
// tiled(), h for 16-bit types is rounded to f16 under a power of two per row.
hipError_t grouped(const MoePlan &p, const void *x, const int32_t *idx, const float *weights, const Q4View &gate,
                   const Q4View &up, const Q4View &down, void *y, int64_t T, int64_t k, int dtype, char *b, hipStream_t s) {
    Q4GroupArgs g{};
    g.w = gate, g.w2 = up, g.x = x, g.y = reinterpret_cast<float *>(b + p.off_h), g.idx = idx, g.weights = weights;
    g.slots = (int)p.slots, g.topk = (int)k;
    hipError_t e = launch_q4_group_gate_up(g, dtype, s);
    if (e != hipSuccess) return e;
    Q4GroupArgs d = g;
    d.w = down, d.x = g.y, d.y = reinterpret_cast<float *>(b + p.off_part);
    e = launch_q4_group_down(d, q4_planes(dtype), s);
    if (e != hipSuccess) return e;
    return sum(d.y, idx, y, T, k, gate.E, down.N, dtype, s);
}

// Few rows per expert: tiles of 16 rows, h in f32.
hipError_t skinny(const MoePlan &p, const void *x, const float *weights, const Q4View &gate, const Q4View &up,
                  const Q4View &down, int64_t k, int dtype, char *b, hipStream_t s) {
    Q4Args g{};
    g.w = gate, g.w2 = up, g.x = x, g.y = b + p.off_h, g.topk = (int)k, g.weights = weights;
    g.ntiles = reinterpret_cast<const int32_t *>(b), g.order = reinterpret_cast<const int32_t *>(b + p.off_order);
    g.tiles = reinterpret_cast<const int4 *>(b + p.off_tiles);
    Q4Args d = g;
    d.w = down, d.x = g.y, d.y = b + p.off_part;
    hipError_t e;
    if (dtype == kF16) e = product<kXF16, kGateUp>(p, g, s);
    else if (dtype == kBF16) e = product<kXBF16, kGateUp>(p, g, s);
    else e = product<kXF32x3, kGateUp>(p, g, s);
    if (e != hipSuccess) return e;
    // h for a 16-bit result is taken in 16 bits (two bfloat16 parts, relative error 2^-17)
    return dtype == kF32 ? product<kXF32x3, kDown>(p, d, s) : product<kXF32x2, kDown>(p, d, s);
}

// Many rows per expert.  For 16-bit types h is rounded to f16 under a power of two per row and
// unit of 128, from its largest value there: half a step of f16 (2^-11 of each value down to 2^-29 of the
// unit's largest) in front of a sum over f, as much as the result's own rounding for f16 and an
// eighth of it for bfloat16; f32 h goes through f32 and two planes.
hipError_t tiled(const MoePlan &p, const void *x, const float *weights, const Q4View &gate, const Q4View &up,
                 const Q4View &down, const Q4Prep &px, int64_t k, int dtype, char *b, hipStream_t s) {
    const int planes = q4_planes(dtype), bm = (int)p.tile_rows;
    const bool plain = q4_plain_x(gate.K, dtype);
    Q4TArgs g{};
    g.w = gate, g.w2 = up, g.topk = (int)k, g.weights = weights, g.y = b + p.off_h, g.ldh = p.ldh;
    g.ntiles = reinterpret_cast<const int32_t *>(b), g.order = reinterpret_cast<const int32_t *>(b + p.off_order);
    g.tiles = reinterpret_cast<const int4 *>(b + p.off_tiles);
    g.a = plain ? static_cast<const _Float16 *>(x) : px.out, g.lda = plain ? gate.K : px.lda, g.plane = px.plane;
    g.rowscale = px.rowscale, g.hexp = reinterpret_cast<int16_t *>(b + p.off_hexp);
    hipError_t e = launch_q4_tiled_gate_up(g, planes, bm, p.max_tiles, s);
    if (e != hipSuccess) return e;
    Q4TArgs d = g;
    d.w = down, d.y = b + p.off_part, d.rowscale = nullptr, d.lda = p.ldh, d.plane = p.slots * p.ldh;
    d.a = reinterpret_cast<const _Float16 *>(b + p.off_h);
    if (dtype == kF32) {
        Q4Prep ph{};
        ph.x = g.y, ph.rows = p.slots, ph.K = gate.N, ph.lda = p.ldh, ph.plane = d.plane;
        ph.out = reinterpret_cast<_Float16 *>(b + p.off_hplanes), ph.rowscale = reinterpret_cast<float *>(b + p.off_hscale);
        e = launch_q4_prep(ph, kF32, s);
        if (e != hipSuccess) return e;
        d.a = ph.out, d.rowscale = ph.rowscale;
    }
    return launch_q4_tiled_down(d, planes, bm, p.max_tiles, s);
}

}  // namespace

// Up to kDirectSlots slots, or up to kDirectSpread while that is no more than one per expert, each reads its
// expert's weights for itself; their rows have to fit in LDS.  (64 experts, 8 each, 2048 x 1024: 40 slots 32 us,
// found by their expert's workgroups 50, 64 slots 45 and 63; of 8 experts, 48 slots 21 and 17.)
// Beyond, by slots per expert (bf16; 64 experts of 8, 2048 x 1024: "large", 8 experts of 2, 1024 x 1024:
// "small", which tiles of the gate product cannot fill the 256 compute units with):
//   up to 8 (4 if small): workgroups find their slots (large, 64 tokens: 93 us, tiles of 64 rows
//     122; small, 33 tokens: 22, rows of 16 20);
//   up to 48, small: plan and blocks of 16 rows (33 tokens 20, tiles of 64 35; 128 tokens 35 and 36);
//   then tiles of 64 rows (large, 128 tokens: 122, found slots 145; 256 tokens 126, rows of 16 207;
//     small, 256 tokens 37, rows of 16 54);
//   from 256 on tiles of 128 (large, 2048 tokens: 392, of 64 408; 1024 tokens 259 and 244).  f32, 598, has
//     tiles of 64 only: its two planes were slower in tiles of 128 (629 against 591).
constexpr int64_t kDirectSlots = 32, kDirectSpread = 64;
constexpr size_t kDirectLds = 48 * 1024;

MoePlan moe_plan(int64_t T, int64_t k, int64_t E, int64_t d, int64_t f, int dtype) {
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    MoePlan p{};
    const bool plain = q4_plain_x(d, dtype), f32 = dtype == kF32;
    p.slots = T * k;
    p.ldx = (d + 127) / 128 * 128, p.ldh = (f + 127) / 128 * 128;
    p.direct = p.slots <= (E < kDirectSlots ? kDirectSlots : E < kDirectSpread ? E : kDirectSpread) && q4_row_lds(p.ldx / 128, f32 ? 3 : 1) <= kDirectLds &&
               q4_row_lds(k * (p.ldh / 128), f32 ? 3 : 2) <= kDirectLds;
    const bool fills = E * ((f + 127) / 128) >= 256;
    const int64_t few = fills ? 8 * E : 4 * E;
    p.grouped = !p.direct && p.slots <= kGroupMaxSlots && p.slots <= few && d <= kGroupMaxK && f <= kGroupMaxK &&
                q4_group_lds(d > f ? d : f, q4_planes(dtype), 16) <= kGroupLds;
    p.tiled = !p.direct && !p.grouped && p.slots > (fills ? 8 * E : 48 * E);
    p.tile_rows = !p.tiled ? 16 : p.slots >= 256 * E && !f32 ? 128 : 64;
    p.max_tiles = p.slots / p.tile_rows + (E < p.slots ? E : p.slots);
    size_t at = 256;  // the first 256 bytes hold the number of tiles
    auto take = [&](size_t n) {
        const size_t off = at;
        at += up(n);
        return off;
    };
    p.off_order = take((size_t)p.slots * 4);
    p.off_tiles = take((size_t)p.max_tiles * 16);
    p.off_h = take((size_t)p.slots * (p.direct ? p.ldh * 6 : p.tiled && !f32 ? p.ldh * 2 : f * 4));
    p.off_part = take((size_t)p.slots * d * 4);
    if (p.tiled) {
        p.off_x = take(plain ? 0 : (size_t)q4_planes(dtype) * T * p.ldx * 2);
        p.off_xscale = take(plain ? 0 : (size_t)T * 4);
        p.off_hexp = take(f32 ? 0 : (size_t)p.slots * (p.ldh / 128) * 2);
        p.off_hscale = take(f32 ? (size_t)p.slots * 4 : 0);
        p.off_hplanes = take(f32 ? (size_t)2 * p.slots * p.ldh * 2 : 0);
    }
    p.total = at;
    return p;
}

hipError_t launch_q4_moe(const MoePlan &p, const void *x, const int32_t *idx, const float *weights, const Q4View &gate,
                         const Q4View &up, const Q4View &down, void *y, int64_t T, int64_t k, int dtype, void *ws,
                         hipStream_t s) {
    char *b = static_cast<char *>(ws);
    if (p.direct) return direct(p, x, idx, weights, gate, up, down, y, T, k, dtype, b, s);
    if (p.grouped) return grouped(p, x, idx, weights, gate, up, down, y, T, k, dtype, b, s);
    int32_t *ntiles = reinterpret_cast<int32_t *>(b), *order = reinterpret_cast<int32_t *>(b + p.off_order);
    int4 *tiles = reinterpret_cast<int4 *>(b + p.off_tiles);
    const float *part = reinterpret_cast<const float *>(b + p.off_part);
    Q4Prep px{};
    if (p.tiled && !q4_plain_x(gate.K, dtype)) {
        px.x = x, px.rows = T, px.K = gate.K, px.lda = p.ldx, px.plane = T * p.ldx;
        px.out = reinterpret_cast<_Float16 *>(b + p.off_x);
        px.rowscale = reinterpret_cast<float *>(b + p.off_xscale);
    }
    const dim3 grid(1 + (unsigned)((px.rows + 15) / 16)), block(1024);
    const int slots = (int)p.slots, rows = (int)p.tile_rows;
    if (dtype == kF32) moe_plan_kernel<kF32, 2><<<grid, block, 0, s>>>(idx, slots, gate.E, rows, order, tiles, ntiles, px);
    else if (dtype == kF16) moe_plan_kernel<kF16, 1><<<grid, block, 0, s>>>(idx, slots, gate.E, rows, order, tiles, ntiles, px);
    else moe_plan_kernel<kBF16, 1><<<grid, block, 0, s>>>(idx, slots, gate.E, rows, order, tiles, ntiles, px);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    e = p.tiled ? tiled(p, x, weights, gate, up, down, px, k, dtype, b, s) : skinny(p, x, weights, gate, up, down, k, dtype, b, s);
    if (e != hipSuccess) return e;
    return sum(part, idx, y, T, k, gate.E, down.N, dtype, s);
}

}  // namespace tq2
