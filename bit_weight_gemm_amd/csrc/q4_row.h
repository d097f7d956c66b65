// Products of single rows with 4-bit weights: the experts' products of a few slots.
//
// A workgroup owns CB column blocks and one row of x (kRowGateUp: a slot's token), or
// the rows of one token's slots (kRowDownSum), whose products it adds up.  The work is a
// list of items, one per slot and unit of 128 k, dealt to the waves in turn.  A wave
// first sends the loads of its first D items' codes, then helps to bring the rows into
// LDS as matrix operands (f32 rows in bfloat16 parts, split once); after one barrier it
// reads them as broadcasts, all 16 rows of the A operand alike, so that its registers are left for
// codes in flight: these products wait for memory, not for the matrix unit.
// Decode, correction and the treatment of infinities are q4_skinny.h's.
//
// Bound by latency: 8 of 64 experts for one token, 2048 x 1024, 6.4-7.5 us for gate and up (16.8 MB of
// codes, 2.2-2.6 TB/s) and 6.0-7.1 for down, of which an empty launch is about two each.
#pragma once

#include "q4_skinny.h"

namespace tq2 {

enum Q4RowMode { kRowGateUp = 0, kRowDownSum = 1 };

struct Q4RowArgs {
    Q4View w;                // kRowGateUp: gate
    const void *x;           // kRowGateUp: x [T][K]; kRowDownSum: h in bfloat16 parts [slots][P][ldh]
    void *y;                 // kRowGateUp: h in bfloat16 parts [slots][PH][ldh]; kRowDownSum: y [T][N]
    const int32_t *idx;      // [T][topk]
    const float *weights;    // [T][topk]
    int64_t ldh;
    int topk;
    Q4View w2;               // kRowGateUp: up
};

// v as P bfloat16 parts (bits) that add up to it, the last of two rounded.
template <int P>
__device__ __forceinline__ void q4_parts(float v, uint16_t *out) {
#pragma unroll
    for (int q = 0; q < P; ++q) {
        if (P == 2 && q == 1) {
            out[q] = __builtin_bit_cast(uint16_t, (__bf16)v);
        } else {
            const uint32_t b = __builtin_bit_cast(uint32_t, v);
            out[q] = (uint16_t)(b >> 16);
            v = __builtin_isfinite(v) ? v - __builtin_bit_cast(float, b & 0xffff0000u) : 0.0f;
        }
    }
}

// XT: the form of x (kXF16, kXBF16, kXF32x3), or of h (kXF32x2, kXF32x3: its parts).
// PH: parts of the h that kRowGateUp writes.  DT: type of y (kRowDownSum).
template <int XT, int G, int CB, int WAVES, int D, int MODE, int PH, int DT>
__global__ __launch_bounds__(WAVES * 64) void q4_row_kernel(Q4RowArgs p) {
    constexpr bool BF = XT != kXF16, EXACT = XT == kXF32x3;
    constexpr int P = XT == kXF32x3 ? 3 : XT == kXF32x2 ? 2 : 1, GPU_ = 128 / G, T = WAVES * 64;
    constexpr int NC = MODE == kRowGateUp ? CB / 2 : CB;
    extern __shared__ __attribute__((aligned(16))) uint16_t xs[];  // [item][P][128]
    __shared__ float red[WAVES][CB * 16];

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, h = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = p.w.K, ku = p.w.ku, row = blockIdx.y;
    const int slot0 = MODE == kRowGateUp ? row : row * p.topk;
    const int items = MODE == kRowGateUp ? ku : p.topk * ku;
    const bool zeros = p.w.zeros != nullptr;
    if (MODE == kRowGateUp) {
        const int e = p.idx[slot0];
        if (e < 0 || e >= p.w.E) return;  // the whole workgroup
    }

    w4 breg[D][CB];
    uint2 sreg[D][CB];
    uint32_t zreg[D][CB];
    float wt[D];  // the slot's weight; 0 with nothing loaded: dropped
    bool live[D];
    auto load = [&](int st, int it) {
        const int j = MODE == kRowGateUp ? 0 : it / ku, u = MODE == kRowGateUp ? it : it % ku;
        const int e = p.idx[slot0 + j];
        live[st] = e >= 0 && e < p.w.E;
        if (!live[st]) return;
        wt[st] = MODE == kRowDownSum ? p.weights[slot0 + j] : 1.0f;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            const Q4View &w = MODE == kRowGateUp && (cb & 1) ? p.w2 : p.w;
            int nb = blockIdx.x * NC + (MODE == kRowGateUp ? cb >> 1 : cb);
            nb = nb < w.nb ? nb : w.nb - 1;  // past the last: not stored
            const int64_t unit = ((int64_t)e * w.nb + nb) * ku + u;
            breg[st][cb] = (w.codes + unit * 64)[lane];
            q4_load_groups<G>(w.scales + unit * (16 * GPU_), zeros ? w.zeros + unit * (16 * GPU_) : nullptr, r, sreg[st][cb],
                              zreg[st][cb]);
        }
    };
    const int n = (items - wave + WAVES - 1) / WAVES;  // this wave's items: wave, wave + WAVES, ...
#pragma unroll
    for (int st = 0; st < D; ++st)
        if (st < n) load(st, wave + WAVES * st);

    // the rows into LDS, eight k at a time
    for (int i = tid; i < items * 16; i += T) {
        const int it = i >> 4, c = i & 15;
        const int j = MODE == kRowGateUp ? 0 : it / ku, k = (MODE == kRowGateUp ? it : it % ku) * 128 + 8 * c;
        w4 v[P];
#pragma unroll
        for (int q = 0; q < P; ++q) v[q] = w4{};
        if (MODE == kRowGateUp) {
            const int64_t at = (int64_t)(row / p.topk) * K + k;
            if (k < K) {
                if constexpr (XT == kXF32x3) {
                    const w4 *x = reinterpret_cast<const w4 *>(static_cast<const float *>(p.x) + at);
                    q4_split<P>(x[0], x[1], v);
                } else {
                    v[0] = *reinterpret_cast<const w4 *>(static_cast<const uint16_t *>(p.x) + at);
                }
            }
        } else {
            const int e = p.idx[slot0 + j];
            if (k < K && e >= 0 && e < p.w.E) {
#pragma unroll
                for (int q = 0; q < P; ++q)
                    v[q] = *reinterpret_cast<const w4 *>(static_cast<const uint16_t *>(p.x) + ((int64_t)(slot0 + j) * P + q) * p.ldh + k);
            }
        }
#pragma unroll
        for (int q = 0; q < P; ++q) *reinterpret_cast<w4 *>(&xs[(it * P + q) * 128 + 8 * c]) = v[q];
    }
    __syncthreads();

    float acc[CB];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) acc[cb] = 0.0f;
    const uint32_t one2 = BF ? 0x3F803F80u : 0x3C003C00u;
    const w4 ones = {one2, one2, one2, one2};
    auto compute = [&](int st, int it) {
        if (!live[st]) return;
        f4 part[CB], sum = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool first = (32 * j) % G == 0, last = (32 * (j + 1)) % G == 0;
            w4 a[P];
#pragma unroll
            for (int q = 0; q < P; ++q) a[q] = *reinterpret_cast<const w4 *>(&xs[(it * P + q) * 128 + 32 * j + 8 * h]);
            if constexpr (!EXACT) {
                if (first) sum = f4{};
#pragma unroll
                for (int q = 0; q < P; ++q) sum = mfma16<BF>(a[q], ones, sum);
            }
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) {
                const float z = (float)((zreg[st][cb] >> (8 * (32 * j / G))) & 255u);
                w4 b;
                if constexpr (EXACT) b = q4_word_exact(breg[st][cb][j], z);
                else b = q4_word16<BF>(breg[st][cb][j]);
                if (first) part[cb] = f4{};
#pragma unroll
                for (int q = 0; q < P; ++q) part[cb] = mfma16<BF>(a[q], b, part[cb]);
                if (last) {
                    const int g = 32 * j / G;
                    const float s = wt[st] * half_bits((g & 2 ? sreg[st][cb].y : sreg[st][cb].x) >> (16 * (g & 1)));
                    acc[cb] += s * (EXACT ? part[cb][0] : part[cb][0] - (16.0f + z) * sum[0]);
                }
            }
        }
    };
    for (int t0 = 0; t0 < n; t0 += D) {
#pragma unroll
        for (int st = 0; st < D; ++st) {
            const int i = t0 + st;
            if (i < n) {
                compute(st, wave + WAVES * i);
                if (i + D < n) load(st, wave + WAVES * (i + D));
            }
        }
    }
    if (h == 0) {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) red[wave][cb * 16 + r] = acc[cb];
    }
    __syncthreads();
    auto total = [&](int at) {
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < WAVES; ++q) v += red[q][at];
        return v;
    };
    const int nn = blockIdx.x * (NC * 16) + tid;
    if constexpr (MODE == kRowGateUp) {
        if (tid >= NC * 16 || nn >= p.w.N) return;
        const int at = (tid >> 4) * 32 + (tid & 15);
        float g = total(at), u = total(at + 16);
        if (!__builtin_isfinite(g) || !__builtin_isfinite(u)) {
            const int e = p.idx[slot0];
            g = q4_slow_row<XT>(p.x, row / p.topk, p.w, e, nn);
            u = q4_slow_row<XT>(p.x, row / p.topk, p.w2, e, nn);
        }
        uint16_t part[PH];
        q4_parts<PH>(g / (1.0f + expf(-g)) * u, part);
#pragma unroll
        for (int q = 0; q < PH; ++q) static_cast<uint16_t *>(p.y)[((int64_t)row * PH + q) * p.ldh + nn] = part[q];
    } else {
        if (tid >= NC * 16 || nn >= p.w.N) return;
        float v = total(tid);
        if (!__builtin_isfinite(v)) {
            v = 0.0f;
#pragma unroll 1
            for (int j = 0; j < p.topk; ++j) {
                const int e = p.idx[slot0 + j];
                if (e < 0 || e >= p.w.E) continue;
                const uint16_t *x = static_cast<const uint16_t *>(p.x) + (int64_t)(slot0 + j) * P * p.ldh;
                const float dot = q4_slow_dot(p.w, e, nn, [&](int k, float (&v8)[8]) {
                    q4_x8<kXBF16>(x, k, v8);
#pragma unroll
                    for (int q = 1; q < P; ++q) {
                        float part[8];
                        q4_x8<kXBF16>(x, q * p.ldh + k, part);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v8[i] += part[i];
                    }
                });
                v += p.weights[slot0 + j] * dot;
            }
        }
        store_from_float<DT>(p.y, (int64_t)row * p.w.N + nn, v);
    }
}

// LDS that a call's rows take.
inline size_t q4_row_lds(int64_t items, int parts) { return (size_t)items * parts * 256; }

template <int XT, int G, int CB, int WAVES, int D, int MODE, int PH, int DT>
inline hipError_t run_q4_row(const Q4RowArgs &a, int64_t rows, hipStream_t s) {
    constexpr int NC = MODE == kRowGateUp ? CB / 2 : CB, P = XT == kXF32x3 ? 3 : XT == kXF32x2 ? 2 : 1;
    const int64_t items = MODE == kRowGateUp ? a.w.ku : (int64_t)a.topk * a.w.ku;
    q4_row_kernel<XT, G, CB, WAVES, D, MODE, PH, DT>
        <<<dim3((unsigned)((a.w.nb + NC - 1) / NC), (unsigned)rows), dim3(WAVES * 64), q4_row_lds(items, P), s>>>(a);
    return hipGetLastError();
}

}  // namespace tq2
