// What a dense 4-bit product does with a finished sum: y = act(v + bias) + residual, in f32.
#pragma once

#include "q4.h"

namespace tq2 {

enum Q4Act { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

struct Q4Epilogue {
    const void *bias;        // [N], nullptr: none
    const void *residual;    // [M][N] in y's type, nullptr: none
    int bias_f32;            // bias is f32, else of y's type
    int act;
};

// The activations' limit at -inf is 0, where their products would be -inf * 0.
__device__ __forceinline__ float q4_activate(int act, float v) {
    if (act == kActNone) return v;
    if (act == kActRelu) return v < 0.0f ? 0.0f : v;
    if (v == -__builtin_inff()) return 0.0f;
    if (act == kActGelu) return 0.5f * v * erfcf(v * -0.70710678f);
    // v sigmoid(t): t = v, or 2 sqrt(2 / pi) (v + 0.044715 v^3) for the form with tanh
    const float t = act == kActSilu ? v : v * __builtin_fmaf(0.0713548163f * v, v, 1.59576912f);
    return v / (1.0f + expf(-t));
}

template <int DT>
__device__ __forceinline__ float q4_epilogue(const Q4Epilogue &e, float v, int n, int64_t at) {
    if (e.bias) v += e.bias_f32 ? static_cast<const float *>(e.bias)[n] : load_as_float<DT>(e.bias, n);
    v = q4_activate(e.act, v);
    return e.residual ? v + load_as_float<DT>(e.residual, at) : v;
}

}  // namespace tq2
