// Launches of the tiled 4-bit products, and x as f16 planes for them.
#include "q4_tiled.h"

namespace tq2 {

namespace {

// One wave per row.  bfloat16 and f32 rows are multiplied by the power of two that
// brings their largest finite value into [2^14, 2^15): bfloat16's 8 bits are then exact
// in f16 down to 2^-32 of the row's largest value, and below that the error is at most 2^-40 of
// it, sixteen bits under the f32 sums' own (2048 x 4096 bf16: 7-9 us, 3.7-4.8 TB/s, as a copy).  f32 rows become hi + lo: 22 bits, the sum of
// two f16 parts, with the same floor.  Past K up to whole units the planes hold zeros.
template <int DT, int P>
__global__ __launch_bounds__(256) void q4_prep_kernel(Q4Prep p) {
    const int lane = threadIdx.x & 63;
    const int64_t row = p.row0 + (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= p.rows) return;
    constexpr int V = DT == kF32 ? 4 : 8;  // elements of a 16-byte piece
    auto piece = [&](int i, float *v) {    // K is a multiple of 32: whole pieces
        const int64_t at = row * p.K + (int64_t)i * V;
        if constexpr (DT == kF32) {
            const f4 x = *reinterpret_cast<const f4 *>(static_cast<const float *>(p.x) + at);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = x[q];
        } else {
            const w4 x = *reinterpret_cast<const w4 *>(static_cast<const uint16_t *>(p.x) + at);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (DT == kBF16) {
                    v[2 * q] = __builtin_bit_cast(float, x[q] << 16);
                    v[2 * q + 1] = __builtin_bit_cast(float, x[q] & 0xffff0000u);
                } else {
                    v[2 * q] = half_bits(x[q]);
                    v[2 * q + 1] = half_bits(x[q] >> 16);
                }
            }
        }
    };
    const int pieces = p.K / V;
    // the first kHold pieces of a lane stay in registers between the two passes
    constexpr int kHold = 8;
    float held[DT == kF16 ? 1 : kHold][V];
    int shift = 0;
    if constexpr (DT != kF16) {
        float most = 0.0f;
        auto look = [&](const float *v) {
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float a = __builtin_fabsf(v[q]);
                most = a > most && a < __builtin_inff() ? a : most;
            }
        };
#pragma unroll
        for (int c = 0; c < kHold; ++c) {
#pragma unroll
            for (int q = 0; q < V; ++q) held[c][q] = 0.0f;
            if (lane + 64 * c < pieces) piece(lane + 64 * c, held[c]);
        }
#pragma unroll
        for (int c = 0; c < kHold; ++c) look(held[c]);
        for (int i = lane + 64 * kHold; i < pieces; i += 64) {
            float v[V];
            piece(i, v);
            look(v);
        }
        for (int o = 1; o < 64; o <<= 1) most = fmaxf(most, __shfl_xor(most, o));
        shift = q4_row_shift(most);
    }
    float norm = 0.0f;
    const int padded = (int)(p.lda / V);
    auto put = [&](int i, const float *v) {
        typedef _Float16 hv __attribute__((ext_vector_type(V)));
        hv a, b;
#pragma unroll
        for (int q = 0; q < V; ++q) {
            const float x = DT == kF16 ? v[q] : __builtin_ldexpf(v[q], shift);
            norm += x * x;
            a[q] = (_Float16)x;
            if constexpr (P == 2) b[q] = __builtin_isfinite(x) ? (_Float16)(x - (float)a[q]) : (_Float16)0.0f;
        }
        if (!p.out) return;
        *reinterpret_cast<hv *>(p.out + row * p.lda + (int64_t)i * V) = a;
        if constexpr (P == 2) *reinterpret_cast<hv *>(p.out + p.plane + row * p.lda + (int64_t)i * V) = b;
    };
    constexpr int kFrom = DT == kF16 ? 0 : kHold;
    if constexpr (DT != kF16) {
#pragma unroll
        for (int c = 0; c < kHold; ++c)
            if (lane + 64 * c < padded) put(lane + 64 * c, held[c]);
    }
    for (int i = lane + 64 * kFrom; i < padded; i += 64) {
        float v[V] = {};
        if (i < pieces) piece(i, v);
        put(i, v);
    }
    if (p.rowscale && lane == 0) p.rowscale[row] = __builtin_ldexpf(1.0f, -shift);
    if (p.norm_exp) {
        for (int o = 1; o < 64; o <<= 1) norm += __shfl_xor(norm, o);
        int e = -200;
        if (norm > 0.0f && norm < __builtin_inff()) {
            (void)__builtin_frexpf(norm, &e);
            e += 1 - 2 * shift;  // one more for the sum's own rounding
        }
        if (lane == 0) p.norm_exp[row] = e;
    }
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

template <int G>
hipError_t dense(const Q4TArgs &a, int dtype, int bm, hipStream_t s) {
    const int64_t t64 = (a.M + 63) / 64, t128 = (a.M + 127) / 128;
    if (dtype == kF32) {
        if constexpr (G > 32)
            if (bm == 128) return run_q4_tiled<128, G, 2, kTDense, kF32>(a, t128, s);
        return run_q4_tiled<64, G, 2, kTDense, kF32>(a, t64, s);  // with G = 32 tiles of 64 only
    }
    if (dtype == kF16) return bm == 64 ? run_q4_tiled<64, G, 1, kTDense, kF16>(a, t64, s) : run_q4_tiled<128, G, 1, kTDense, kF16>(a, t128, s);
    return bm == 64 ? run_q4_tiled<64, G, 1, kTDense, kBF16>(a, t64, s) : run_q4_tiled<128, G, 1, kTDense, kBF16>(a, t128, s);
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
    if (a.w.G == 32) return dense<32>(a, dtype, bm, s);
    if (a.w.G == 64) return dense<64>(a, dtype, bm, s);
    return dense<128>(a, dtype, bm, s);
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
