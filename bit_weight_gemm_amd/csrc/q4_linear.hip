// Dense 4-bit products with bias, activation and residual in their epilogue: q4_gemm's kernels and choice among
// them, the epilogue where a sum is finished (the last store, or the join of shares).
#include "q4_skinny.h"
#include "q4_tiled.h"

namespace tq2 {

namespace {

// The shares' sums in their order, as q4_join_kernel, then the epilogue.
template <int DT>
__global__ __launch_bounds__(256) void q4_join_epilogue_kernel(const float *part, int64_t stride, int split, void *y, int64_t n,
                                                               int N, Q4Epilogue epi) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    f4 v = *reinterpret_cast<const f4 *>(part + i);  // the stride leaves room for the last four
    for (int q = 1; q < split; ++q) v += *reinterpret_cast<const f4 *>(part + q * stride + i);
    int col = (int)(i % N);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (i + q < n) store_from_float<DT>(y, i + q, q4_epilogue<DT>(epi, v[q], col, i + q));
        if (++col == N) col = 0;
    }
}

}  // namespace

hipError_t launch_q4_dense_epilogue(const Q4Args &a, int dtype, hipStream_t s) { return q4_dense<true>(a, dtype, s); }

hipError_t launch_q4_tiled_epilogue(const Q4TArgs &a, int dtype, int bm, hipStream_t s) {
    return q4_tiled_dense<true>(a, dtype, bm, s);
}

hipError_t launch_q4_join_epilogue(const Q4TArgs &a, void *y, int dtype, hipStream_t s) {
    const int64_t n = a.M * a.w.N;
    const dim3 grid((unsigned)((n + 1023) / 1024)), block(256);
    if (dtype == kF32) q4_join_epilogue_kernel<kF32><<<grid, block, 0, s>>>(a.part, a.part_stride, a.split, y, n, a.w.N, a.epi);
    else if (dtype == kF16) q4_join_epilogue_kernel<kF16><<<grid, block, 0, s>>>(a.part, a.part_stride, a.split, y, n, a.w.N, a.epi);
    else q4_join_epilogue_kernel<kBF16><<<grid, block, 0, s>>>(a.part, a.part_stride, a.split, y, n, a.w.N, a.epi);
    return hipGetLastError();
}

}  // namespace tq2
