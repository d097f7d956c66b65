// Launches of the tiled 4-bit products, and x as f16 planes for them.
#include "q4_prep.h"

namespace tq2 {

namespace {

template <int DT, int P>
__global__ __launch_bounds__(256) void q4_prep_kernel(Q4Prep p) {
    const int64_t row = p.row0 + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row < p.rows) q4_prep_row<DT, P>(p, row);
}

// y = the sum of the shares' sums, in their order.
template <int DT>
__global__ __launch_bounds__(256) void q4_join_kernel(const float *part, int64_t stride, int split, void *y, int64_t n) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    f4 v = *reinterpret_cast<const f4 *>(part + i);  // the stride leaves room for the last four
    for (int q = 1; q < split; ++q) v += *reinterpret_cast<const f4 *>(part + q * stride + i);
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (i + q < n) store_from_float<DT>(y, i + q, v[q]);
}

template <int G, int MODE>
hipError_t grouped(const Q4TArgs &a, int planes, int bm, int64_t tiles, hipStream_t s) {
    if (planes == 2) return run_q4_tiled<64, G, 2, MODE, kF32>(a, tiles, s);  // tiles of 64 only
    return bm == 64 ? run_q4_tiled<64, G, 1, MODE, kF32>(a, tiles, s) : run_q4_tiled<128, G, 1, MODE, kF32>(a, tiles, s);
}

}  // namespace

hipError_t launch_q4_prep(Q4Prep p, int dtype, hipStream_t s) {
    constexpr int64_t kMost = (int64_t)1 << 25;  // rows of one launch: fewer than 2^32 work items, 64 a row
    for (p.row0 = 0; p.row0 < p.rows; p.row0 += kMost) {
        const int64_t n = p.rows - p.row0 < kMost ? p.rows - p.row0 : kMost;
        const dim3 grid((unsigned)((n + 3) / 4)), block(256);
        if (dtype == kF32) q4_prep_kernel<kF32, 2><<<grid, block, 0, s>>>(p);
        else if (dtype == kF16) q4_prep_kernel<kF16, 1><<<grid, block, 0, s>>>(p);
        else q4_prep_kernel<kBF16, 1><<<grid, block, 0, s>>>(p);
    }
    return hipGetLastError();
}

hipError_t launch_q4_tiled_dense(const Q4TArgs &a, int dtype, int bm, hipStream_t s) {
    return q4_tiled_dense<false>(a, dtype, bm, s);
}

hipError_t launch_q4_join(const float *part, int64_t stride, int split, void *y, int64_t n, int dtype, hipStream_t s) {
    const dim3 grid((unsigned)((n + 1023) / 1024)), block(256);
    if (dtype == kF32) q4_join_kernel<kF32><<<grid, block, 0, s>>>(part, stride, split, y, n);
    else if (dtype == kF16) q4_join_kernel<kF16><<<grid, block, 0, s>>>(part, stride, split, y, n);
    else q4_join_kernel<kBF16><<<grid, block, 0, s>>>(part, stride, split, y, n);
    return hipGetLastError();
}

hipError_t launch_q4_tiled_gate_up(const Q4TArgs &a, int planes, int bm, int64_t tiles, hipStream_t s) {
    if (a.w.G == 32) return grouped<32, kTGateUp>(a, planes, bm, tiles, s);
    if (a.w.G == 64) return grouped<64, kTGateUp>(a, planes, bm, tiles, s);
    return grouped<128, kTGateUp>(a, planes, bm, tiles, s);
}

hipError_t launch_q4_tiled_down(const Q4TArgs &a, int planes, int bm, int64_t tiles, hipStream_t s) {
    if (a.w.G == 32) return grouped<32, kTDown>(a, planes, bm, tiles, s);
    if (a.w.G == 64) return grouped<64, kTDown>(a, planes, bm, tiles, s);
    return grouped<128, kTDown>(a, planes, bm, tiles, s);
}

}  // namespace tq2
