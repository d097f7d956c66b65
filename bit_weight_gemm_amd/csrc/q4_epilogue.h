// What a dense 4-bit product does with a finished sum: y = act(v + bias) + residual, in f32.
#pragma once

#include <type_traits>

#include "q4.h"

namespace tq2 {

enum Q4Act { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

struct Q4Epilogue {
    const void *bias;        // [N], nullptr: none
    const void *residual;    // [M][N] in y's type, nullptr: none
    int bias_f32;            // bias is f32, else of y's type
    int act;
};

// The three that are v times a sigmoid-like factor tend to 0 at -inf, where the product would be -inf * 0.
// For 16-bit results (SHORT) from the hardware's exp2 and reciprocal.  Relative errors, with the steps rounded to f32: below 2^-17 from
// v = -6 on; below, where results are under 1e-8 (gelu) and 1e-10 (its form with tanh), the rounding of the exponent counts more: up
// to 2^-16.6 and 2^-15.9 at -14 (silu 2^-19.9).  An f16 half step is 2^-11, a bf16 one 2^-8.
// gelu is then v Phi(v) with Phi(-a) = e^(-a^2/2) erfcx(a / sqrt 2) / 2 (a = |v|), the second factor a polynomial in 1 / (1 + 0.31 a)
// fitted to least relative error on 0 .. 14.5 (2^-17.7; beyond, e^(-a^2/2) is 0).  What is v times a factor below f32's normal
// range may come out as 0.
template <int ACT, bool SHORT>
__device__ __forceinline__ float q4_act(float v) {
    if constexpr (ACT == kActNone) return v;
    if constexpr (ACT == kActRelu) return v < 0.0f ? 0.0f : v;
    float out;
    if constexpr (ACT == kActGelu && SHORT) {
        const float a = __builtin_fabsf(v), t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.31f, a, 1.0f));
        float h = __builtin_fmaf(t, -0.07392820715904236f, 0.18044771254062653f);
        h = __builtin_fmaf(t, h, 0.01574752666056156f);
        h = __builtin_fmaf(t, h, 0.13342836499214172f);
        h = __builtin_fmaf(t, h, 0.12044161558151245f);
        h = __builtin_fmaf(t, h, 0.1238606721162796f);
        h *= t * __builtin_amdgcn_exp2f(v * v * -0.72134752f);
        out = v * (v < 0.0f ? h : 1.0f - h);
    } else if constexpr (ACT == kActGelu) {
        out = 0.5f * v * erfcf(v * -0.70710678f);
    } else {
        // v sigmoid(t): t = v, or 2 sqrt(2 / pi) (v + 0.044715 v^3) for the form with tanh
        const float t = ACT == kActSilu ? v : v * __builtin_fmaf(0.0713548163f * v, v, 1.59576912f);
        if constexpr (SHORT) out = v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t * -1.44269504f));
        else out = v / (1.0f + expf(-t));
    }
    return v < -1e30f ? 0.0f : out;
}

// Of n values, by one look at the activation.
template <bool SHORT, int N>
__device__ __forceinline__ void q4_activate(int act, float (&v)[N]) {
    auto all = [&](auto kind) {
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = q4_act<decltype(kind)::value, SHORT>(v[q]);
    };
    if (act == kActRelu) all(std::integral_constant<int, kActRelu>{});
    else if (act == kActGelu) all(std::integral_constant<int, kActGelu>{});
    else if (act == kActGeluTanh) all(std::integral_constant<int, kActGeluTanh>{});
    else if (act == kActSilu) all(std::integral_constant<int, kActSilu>{});
}

// An element's bits as loaded, and their value: apart, so that nothing waits for the load until the value is used.
template <int DT>
__device__ __forceinline__ uint32_t q4_bits(const void *p, int64_t i) {
    if constexpr (DT == kF32) return static_cast<const uint32_t *>(p)[i];
    return static_cast<const uint16_t *>(p)[i];
}
template <int DT>
__device__ __forceinline__ float q4_value(uint32_t bits) {
    if constexpr (DT == kF32) return __builtin_bit_cast(float, bits);
    if constexpr (DT == kF16) return half_bits(bits);
    return __builtin_bit_cast(float, bits << 16);
}
template <int DT>
__device__ __forceinline__ uint32_t q4_bias_bits(const Q4Epilogue &e, int n) {
    if (!e.bias) return 0;
    return e.bias_f32 ? q4_bits<kF32>(e.bias, n) : q4_bits<DT>(e.bias, n);
}
template <int DT>
__device__ __forceinline__ float q4_bias_value(const Q4Epilogue &e, uint32_t bits) {
    return e.bias_f32 ? q4_value<kF32>(bits) : q4_value<DT>(bits);
}
template <int DT>
__device__ __forceinline__ uint32_t q4_residual_bits(const Q4Epilogue &e, int64_t at) {
    return e.residual ? q4_bits<DT>(e.residual, at) : 0;
}
// bits: of the bias and the residual.
template <int DT>
__device__ __forceinline__ float q4_epilogue(const Q4Epilogue &e, float v, uint32_t bias, uint32_t residual) {
    float one[1] = {v + q4_bias_value<DT>(e, bias)};
    q4_activate<DT != kF32>(e.act, one);
    return one[0] + q4_value<DT>(residual);
}
template <int DT>
__device__ __forceinline__ float q4_epilogue(const Q4Epilogue &e, float v, int n, int64_t at) {
    return q4_epilogue<DT>(e, v, q4_bias_bits<DT>(e, n), q4_residual_bits<DT>(e, at));
}

}  // namespace tq2
