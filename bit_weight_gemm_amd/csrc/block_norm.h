// Rows in registers and their sums: what the norms of a block and a mixture layer's router share (gfx950).
#pragma once

#include "pieces.h"

namespace tq2 {

// ---- sums over a wave or a workgroup, the same bits in every lane

template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_mov_dpp((int)b, CTRL, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// v of both lanes of each exchanged pair, added
__device__ __forceinline__ double add16(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const auto l = __builtin_amdgcn_permlane16_swap((unsigned)b, (unsigned)b, false, false);
    const auto h = __builtin_amdgcn_permlane16_swap((unsigned)(b >> 32), (unsigned)(b >> 32), false, false);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)h[0] << 32 | (uint32_t)l[0]) +
           __builtin_bit_cast(double, (uint64_t)(uint32_t)h[1] << 32 | (uint32_t)l[1]);
}
__device__ __forceinline__ double add32(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const auto l = __builtin_amdgcn_permlane32_swap((unsigned)b, (unsigned)b, false, false);
    const auto h = __builtin_amdgcn_permlane32_swap((unsigned)(b >> 32), (unsigned)(b >> 32), false, false);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)h[0] << 32 | (uint32_t)l[0]) +
           __builtin_bit_cast(double, (uint64_t)(uint32_t)h[1] << 32 | (uint32_t)l[1]);
}
__device__ __forceinline__ double wave_total(double v) {
    v += dpp64<0xB1>(v);   // lane ^ 1
    v += dpp64<0x4E>(v);   // lane ^ 2
    v += dpp64<0x141>(v);  // mirrored in eight lanes
    v += dpp64<0x140>(v);  // mirrored in sixteen
    return add32(add16(v));
}

// Sums of v[0 .. K-1] over the TPR threads of a row (whole waves; TPR 64: the wave's own).  `room` [TPR / 64][K] is
// another one at each of two sums in a row, so that one barrier is enough.
template <int TPR, int K>
__device__ __forceinline__ void row_total(double (&v)[K], double *room) {
#pragma unroll
    for (int q = 0; q < K; ++q) v[q] = wave_total(v[q]);
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int q = 0; q < K; ++q) room[wave * K + q] = v[q];
        __syncthreads();
#pragma unroll
        for (int q = 0; q < K; ++q) {
            double s = 0;
#pragma unroll
            for (int w = 0; w < TPR / 64; ++w) s += room[w * K + q];
            v[q] = s;
        }
    }
}

// v rounded to type DT.
template <int DT>
__device__ __forceinline__ float rounded(float v) {
    if constexpr (DT == kF32) return v;
    else if constexpr (DT == kF16) return (float)(_Float16)v;
    else return (float)(__bf16)v;
}

// ---- a row's norm

// Mean and 1 / standard deviation from the sums of N values and of their squares (rms: mean 0).  In f64: the roundings of a
// normed row, which decide experts where a router follows, are those of its exact value but for one in some 2^28 (a sum in another
// order would give another 2^-24).  The variance is a difference: its relative error is some 2^-47 (mean / deviation)^2, so it is good
// for means of up to kFarMean deviations.  Callers whose rows may lie farther away subtract a mean first, or sum again (is_far).
struct Norm {
    double mean, rstd;
};
constexpr double kFarMean = 1024.0;
__device__ __forceinline__ bool is_far(const Norm &r) { return __builtin_fabs(r.mean) * r.rstd > kFarMean; }
__device__ __forceinline__ Norm norm_of(double sum, double squares, int N, bool layer, double eps) {
    Norm r;
    r.mean = layer ? sum / N : 0.0;
    const double var = squares / N - r.mean * r.mean;
    r.rstd = 1.0 / sqrt((var < 0.0 ? 0.0 : var) + eps);
    return r;
}
// (without FULL no mean, and no bias)
template <bool FULL>
__device__ __forceinline__ float norm_value(const Norm &r, float v, float weight, float bias) {
    float f;
    if constexpr (FULL) f = (float)(((double)v - r.mean) * r.rstd * (double)weight + (double)bias);
    else f = (float)((double)v * r.rstd * (double)weight);
    // rounded here, and again to the rows' type: the compiler would make one rounding of both, whose results differ from
    // the two's (and from a cast through f32) in one f16 value of some 2^14, at twenty more instructions
    asm("" : "+v"(f));
    return f;
}

// ---- launchers (arguments checked by the C ABI layer)

struct BlockNormArgs {
    const void *x, *b;               // [M][N]; b may be null: y is x
    const void *post, *post_bias;    // [N] or null
    const void *gate;                // [R][N] or null
    const void *pre, *pre_bias;      // [N] or null
    void *y, *n;                     // [M][N] or null
    int64_t M, gate_rows;            // rows that share a gate: M / R
    int N;
    bool layer;
    float scale;
    double eps;
};
hipError_t launch_block_norm(const BlockNormArgs &a, int dtype, bool wide_weights, hipStream_t s);

struct BlockNormBackwardArgs {
    const void *dy, *dn, *y, *b;     // [M][N]; null: none
    const void *post, *post_bias, *gate, *pre, *pre_bias;
    void *dx, *db;                   // [M][N]; db null: no b
    float *dpost, *dpost_bias, *dgate, *dpre, *dpre_bias;  // null: not asked for
    float *part;                     // workspace
    int64_t M, gate_rows;
    int N;
    bool layer;
    float scale;
    double eps;
};
size_t block_norm_backward_workspace(int64_t M, int64_t N, int64_t R, int dtype);
hipError_t launch_block_norm_backward(const BlockNormBackwardArgs &a, int dtype, bool wide_weights, void *ws, hipStream_t s);

}  // namespace tq2
