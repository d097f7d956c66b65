// 4-bit weights under group scales: packed layout, views and in-register decode (gfx950).
//
// A weight W[n][k] = (code - zero) * scale has 4-bit codes, one f16 scale and one
// zero point (8 where none are given) per row and group of G = 32, 64 or 128
// consecutive k.  Weights of several experts are stacked.
//
// Packed layout (built on the GPU by q4_pack), for E experts, NB = ceil(N/16)
// blocks of 16 rows and KU = ceil(K/128) units of 128 k:
//   codes  : 16 bytes [E][NB][KU][64 lanes].  Lane l of a unit holds row l%16 of the
//            block; word j of its 16 bytes holds the eight codes k = 128u + 32j +
//            8(l/16) .. +7, which is lane l's B operand of the j-th
//            v_mfma_f32_16x16x32 of the unit: a wave reads a unit as one
//            contiguous kilobyte, straight into the registers it decodes from.
//            Inside a word element e sits at bits 4(e>>1) + 16(e&1), so that one
//            shift and one masked insert give a pair of consecutive k as two halves.
//   scales : f16 [E][NB][KU][16 rows][128/G]
//   zeros  : u8, the same order (absent when every zero point is 8)
// Rows past N and groups past K have scale 0 and code 0.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode.h"

namespace tq2 {

typedef uint32_t w4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

enum Q4Type { kF32 = 0, kF16 = 1, kBF16 = 2 };

// Bytes before the codes: unused, kept so that packed weights that a program stored keep their layout.
inline size_t q4_head_bytes(int64_t E) { return (size_t)(E * 4 + 255) / 256 * 256; }

struct Q4Layout {
    int64_t nb, ku;                          // row blocks and units of one expert
    size_t codes_off, scales_off, zeros_off, total;
};

inline Q4Layout q4_layout(int64_t E, int64_t N, int64_t K, int64_t G, bool zeros) {
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    Q4Layout L{};
    L.nb = (N + 15) / 16;
    L.ku = (K + 127) / 128;
    const size_t units = (size_t)E * L.nb * L.ku, groups = units * 16 * (128 / G);
    L.codes_off = q4_head_bytes(E);
    L.scales_off = L.codes_off + units * 1024;
    L.zeros_off = L.scales_off + up(groups * 2);
    L.total = L.zeros_off + (zeros ? up(groups) : 0);
    return L;
}

// What the kernels take of a packed weight.
struct Q4View {
    const w4 *codes;
    const uint16_t *scales;
    const uint8_t *zeros;    // nullptr: every zero point is 8
    int E, N, K, G, nb, ku;
};

inline Q4View q4_view(const void *data, int64_t E, int64_t N, int64_t K, int64_t G, bool zeros) {
    const Q4Layout L = q4_layout(E, N, K, G, zeros);
    const char *b = static_cast<const char *>(data);
    Q4View v{};
    v.codes = reinterpret_cast<const w4 *>(b + L.codes_off);
    v.scales = reinterpret_cast<const uint16_t *>(b + L.scales_off);
    v.zeros = zeros ? reinterpret_cast<const uint8_t *>(b + L.zeros_off) : nullptr;
    v.E = (int)E, v.N = (int)N, v.K = (int)K, v.G = (int)G, v.nb = (int)L.nb, v.ku = (int)L.ku;
    return v;
}

// Eight codes as 16 + code in f16 (BF: bfloat16): both formats have an exponent at
// which the code fits the fraction exactly (f16 0x4C00 | code << 6, bfloat16 0x4180
// | code << 3).  A shift and a masked insert per pair, eight instructions a word,
// against nine for the exact code - zero in f16 and about twenty in bfloat16, which
// has no packed arithmetic.  The 16 + zero is taken off each group's sum:
//   sum x (code - zero) = sum x (16 + code) - (16 + zero) sum x,
// with sum x from the same matrix instructions against a column of ones.
template <bool BF>
__device__ __forceinline__ w4 q4_word16(uint32_t w) {
    if constexpr (BF) {
        constexpr uint32_t m = 0x00780078u, one = 0x41804180u;
        return w4{((w << 3) & m) | one, ((w >> 1) & m) | one, ((w >> 5) & m) | one, ((w >> 9) & m) | one};
    } else {
        constexpr uint32_t m = 0x03C003C0u, one = 0x4C004C00u;
        return w4{((w << 6) & m) | one, ((w << 2) & m) | one, ((w >> 2) & m) | one, ((w >> 6) & m) | one};
    }
}

// The eight code - zero of a word in bfloat16, exact (zf: the zero point as a float):
// codes to floats by byte, and the upper halves of the differences.  Twenty-odd
// instructions; for f32 x, where the correction's larger terms would show.
__device__ __forceinline__ w4 q4_word_exact(uint32_t w, float zf) {
    const uint32_t a = w & 0x0F0F0F0Fu, b = (w >> 4) & 0x0F0F0F0Fu;  // bytes: elements 0 4 1 5, and 2 6 3 7
    auto pair = [&](uint32_t v, int lo, int hi) {
        const float x = (float)((v >> (8 * lo)) & 255u) - zf, y = (float)((v >> (8 * hi)) & 255u) - zf;
        return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, y), __builtin_bit_cast(uint32_t, x), 0x07060302u);
    };
    return w4{pair(a, 0, 2), pair(b, 0, 2), pair(a, 1, 3), pair(b, 1, 3)};
}

template <bool BF>
__device__ __forceinline__ f4 mfma16(w4 a, w4 b, f4 c) {
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

// v is computed by this point of the program (no instruction).
__device__ __forceinline__ void q4_here(f4 &v) { asm volatile("" : "+v"(v)); }

__device__ __forceinline__ float half_bits(uint32_t h) { return (float)__builtin_bit_cast(_Float16, (uint16_t)h); }

// Row r's scales (f16, the first in the low half of .x) and zero points (a byte each; 8
// where zeros is null) in a unit, from the unit's places (uniform in a wave): 128/G of them.
template <int G>
__device__ __forceinline__ void q4_load_groups(const uint16_t *scales, const uint8_t *zeros, int r, uint2 &s, uint32_t &z) {
    if constexpr (G == 128) s.x = scales[r];
    if constexpr (G == 64) s.x = reinterpret_cast<const uint32_t *>(scales)[r];
    if constexpr (G == 32) s = reinterpret_cast<const uint2 *>(scales)[r];
    z = 0x08080808u;
    if (zeros) {
        if constexpr (G == 128) z = zeros[r];
        if constexpr (G == 64) z = reinterpret_cast<const uint16_t *>(zeros)[r];
        if constexpr (G == 32) z = reinterpret_cast<const uint32_t *>(zeros)[r];
    }
}

template <int DT>
__device__ __forceinline__ float load_as_float(const void *p, int64_t i) {
    if constexpr (DT == kF32) return static_cast<const float *>(p)[i];
    if constexpr (DT == kF16) return (float)static_cast<const _Float16 *>(p)[i];
    return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
}

// Stores round to nearest even.
template <int DT>
__device__ __forceinline__ void store_from_float(void *p, int64_t i, float v) {
    if constexpr (DT == kF32) static_cast<float *>(p)[i] = v;
    else if constexpr (DT == kF16) static_cast<_Float16 *>(p)[i] = (_Float16)v;
    else static_cast<__bf16 *>(p)[i] = (__bf16)v;
}

// Code of element (n, k) of expert e, and its scale and zero point (scalar form).
__device__ __forceinline__ float q4_weight_at(const Q4View &w, int e, int n, int k) {
    const int64_t unit = ((int64_t)e * w.nb + (n >> 4)) * w.ku + (k >> 7);
    const uint32_t word = w.codes[unit * 64 + ((k & 31) >> 3) * 16 + (n & 15)][(k & 127) >> 5];
    const int el = k & 7;
    const int code = (word >> (4 * (el >> 1) + 16 * (el & 1))) & 15;
    const int64_t g = (unit * 16 + (n & 15)) * (128 / w.G) + (k & 127) / w.G;
    const int zero = w.zeros ? w.zeros[g] : 8;
    return (float)(code - zero) * half_bits(w.scales[g]);
}

// ---- launchers (arguments checked by the C ABI layer)

hipError_t launch_q4_pack(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, const Q4View &v,
                          hipStream_t s);
hipError_t launch_q4_dequant(const Q4View &v, float *out, hipStream_t s);
size_t q4_gemm_workspace(int64_t N, int64_t K, int64_t G, int64_t M, int dtype);
hipError_t launch_q4_gemm(const Q4View &v, const void *x, void *y, int64_t M, int dtype, void *ws, hipStream_t s);

// Experts' products.  Workspace: see MoePlan.
struct MoePlan {
    int64_t slots;                   // T * k
    bool direct;                     // a few slots: no plan
    bool grouped;                    // a few rows per expert: no plan either
    bool tiled;                      // many rows per expert: the tiled products
    int64_t tile_rows, max_tiles;    // rows per tile of the grouped products, and the most tiles there can be
    int64_t ldx, ldh;                // tiled: rows of x and of h in whole units of 128
    size_t off_order, off_tiles, off_h, off_part, off_x, off_xscale, off_hexp, off_hscale, off_hplanes, total;
};
MoePlan moe_plan(int64_t T, int64_t k, int64_t E, int64_t d, int64_t f, int dtype);
hipError_t launch_q4_moe(const MoePlan &p, const void *x, const int32_t *idx, const float *weights, const Q4View &gate,
                         const Q4View &up, const Q4View &down, void *y, int64_t T, int64_t k, int dtype, void *ws,
                         hipStream_t s);

struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *idx;
    float *weights;
    int64_t T;
    int E, k, groups, keep, group_top, dtype;
    int n;                   // experts per group (set by the launcher)
    bool sigmoid, renorm;
};
hipError_t launch_moe_route(const RouteArgs &a, hipStream_t s);
hipError_t launch_moe_route_backward(const void *logits, const int32_t *idx, const float *dw, void *dlogits, int64_t T,
                                     int E, int k, int dtype, bool sigmoid, bool renorm, hipStream_t s);

}  // namespace tq2
