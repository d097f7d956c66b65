// x as f16 planes for the tiled products.
#pragma once

#include "q4_tiled.h"

namespace tq2 {

// One wave per row.  bfloat16 and f32 rows are multiplied by the power of two that
// brings their largest finite value into [2^14, 2^15): bfloat16's 8 bits are then exact
// in f16 down to 2^-31 of the row's largest value, and below that the error is at most
// 2^-39 of it, fifteen bits under the f32 sums' own.  f32 rows become hi + lo: 22 bits, the
// sum of two f16 parts, with the same floor.  Past K up to whole units the planes hold
// zeros.  2048 x 4096 bf16: 7-9 us, 3.7-4.8 TB/s, as a copy.
template <int DT, int P>
__device__ void q4_prep_row(const Q4Prep &p, int64_t row) {
    const int lane = threadIdx.x & 63;
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
    const int padded = (int)(p.lda / V);
    auto put = [&](int i, const float *v) {
        typedef _Float16 hv __attribute__((ext_vector_type(V)));
        hv a, b;
#pragma unroll
        for (int q = 0; q < V; ++q) {
            const float x = DT == kF16 ? v[q] : __builtin_ldexpf(v[q], shift);
            a[q] = (_Float16)x;
            if constexpr (P == 2) b[q] = __builtin_isfinite(x) ? (_Float16)(x - (float)a[q]) : (_Float16)0.0f;
        }
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
    if (lane == 0) p.rowscale[row] = __builtin_ldexpf(1.0f, -shift);
}

}  // namespace tq2
