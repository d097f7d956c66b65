// Products of few rows with a 4-bit weight: y[m][n] = sum_k x[m][k] (code - zero) scale.
//
// A wave owns CB blocks of 16 output columns and RB blocks of 16 rows.  WK of a
// workgroup's eight waves share them and take the 128-k units in turn (the w-th the units
// w, w + WK, ...), so at each turn they read adjacent units of a column block; the
// others have the next columns.  A wave loads a unit's codes as one contiguous kilobyte
// per column block and its x straight into the A operand's registers (lane l: row
// l%16, k = 32j + 8(l/16) .. +7): nothing goes through LDS and no wave waits for
// another until the WK partial tiles are added, in wave order, at the end.  Both
// streams run D units ahead.  WK is the smallest that gives the chip eight waves per
// compute unit: a wave that has one unit only spends its time on its first loads.
//
// The codes are decoded to 16 + code (q4_word16); each group's sum is corrected and
// scaled in f32: acc += scale (part - (16 + zero) S), with S = sum x over the group
// from a matrix instruction against ones.  The products are exact and the sums f32;
// the correction's terms are at most 31/15 times as large as the largest weight's,
// so it costs about two bits of the f32 sum and none of the result's.
//
// For f32 x the codes are decoded to code - zero itself, so that no term is larger
// than the product's own (relative error of a 23 x 5003 x 4000 product 2e-7; with the
// correction 1e-6).
//
// x is used as it is where it is f16 or bfloat16.  f32 x is split into three
// bfloat16 parts that add up to it exactly (kXF32x3), or for an intermediate whose
// consumer rounds to 16 bits into two (kXF32x2: 16 bits kept, relative error 2^-17).
//
// An output that comes out infinite or NaN is formed again term by term
// (q4_slow_dot): the correction makes Inf - Inf of an infinite x, where the sum itself
// may be an infinity of one sign.
//
// Bound by the loads' latency and their number in flight: one row, 4096 x 4096, bf16, 3.7-4.8 us of
// kernel (2 TB/s; a copy of gigabytes reaches 4.8), eight rows, 14336 x 4096, G = 32, f16, 11-12 us
// (3.1 TB/s); 23 f32 rows, 5003 x 4000, 17 us, where the split of x and the exact decode
// count.  Rows that M does not have are not loaded (eight rows 12.5 -> 11.3 us).
#pragma once

#include "q4.h"

namespace tq2 {

enum Q4X { kXF16 = 0, kXBF16 = 1, kXF32x2 = 2, kXF32x3 = 3 };
// kDense: y = x W^T in x's type.  kGateUp: h[p][n] = silu(g) u of the slot at sorted
// place p (f32).  kDown: part[slot][n] = weight[slot] * (h W^T) (f32).
enum Q4Mode { kDense = 0, kGateUp = 1, kDown = 2 };

// What every launch reads comes first: in the argument block's first two lines of 64 bytes (behind w2, eight
// rows of 14336 x 4096 took 11.47 us, so 11.29).
struct Q4Args {
    Q4View w;                // kGateUp: gate
    const void *x;
    void *y;
    int64_t M;               // kDense: rows of x
    int topk;                // slots per token
    int log_wk;              // waves that share a column block: 1 << log_wk
    Q4View w2;               // kGateUp: up
    const int32_t *order;    // slots sorted by expert
    const int4 *tiles;       // {expert, first place, rows, 0}
    const int32_t *ntiles;
    const float *weights;    // [slots]
};

// sum_k x[k] W[n][k] of expert e term by term, k in order, eight at a time: one word of codes, x8(k) for the
// values of x there.  One row of 4096 x 4096 with an infinity 145 us, with a NaN 7 to 145 by its place (an element
// at a time 700).
template <typename X>
__device__ __forceinline__ float q4_slow_dot(const Q4View &w, int e, int n, X &&x8) {
    const int r = n & 15, groups = 128 / w.G;
    const int64_t unit0 = ((int64_t)e * w.nb + (n >> 4)) * w.ku;
    float acc = 0.0f;
#pragma unroll 1
    for (int k = 0; k < w.K && acc == acc; k += 8) {  // (NaN stays NaN)
        const int64_t unit = unit0 + (k >> 7);
        const uint32_t word = reinterpret_cast<const uint32_t *>(w.codes + unit * 64 + ((k & 31) >> 3) * 16 + r)[(k & 127) >> 5];
        const int64_t at = (unit * 16 + r) * groups + (k & 127) / w.G;
        const float scale = half_bits(w.scales[at]), zero = w.zeros ? (float)w.zeros[at] : 8.0f;
        float x[8];
        x8(k, x);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc += x[q] * (((float)((word >> (4 * (q >> 1) + 16 * (q & 1))) & 15u) - zero) * scale);
    }
    return acc;
}

// Eight values of a row of x at k.
template <int XT>
__device__ __forceinline__ void q4_x8(const void *x, int64_t at, float (&v)[8]) {
    if constexpr (XT == kXF16 || XT == kXBF16) {
        const w4 b = *reinterpret_cast<const w4 *>(static_cast<const uint16_t *>(x) + at);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint32_t bits = q & 1 ? b[q >> 1] >> 16 : b[q >> 1] & 0xffffu;
            v[q] = XT == kXF16 ? half_bits(bits) : __builtin_bit_cast(float, bits << 16);
        }
    } else {
        const f4 *p = reinterpret_cast<const f4 *>(static_cast<const float *>(x) + at);
        const f4 a = p[0], b = p[1];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = a[q], v[4 + q] = b[q];
    }
}
template <int XT>
__device__ __forceinline__ float q4_slow_row(const void *x, int64_t row, const Q4View &w, int e, int n) {
    return q4_slow_dot(w, e, n, [&](int k, float (&v)[8]) { q4_x8<XT>(x, row * w.K + k, v); });
}

// Eight floats as P bfloat16 parts: each part is cut, so that what is left is exact,
// except the last of two, which is rounded to nearest even.
template <int P>
__device__ __forceinline__ void q4_split(w4 lo, w4 hi, w4 *out) {
    uint32_t v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t &a = v[2 * i], &b = v[2 * i + 1];
            if (P == 2 && q == 1) {
                typedef __bf16 b2 __attribute__((ext_vector_type(2)));
                const b2 t = {(__bf16)__builtin_bit_cast(float, a), (__bf16)__builtin_bit_cast(float, b)};
                out[q][i] = __builtin_bit_cast(uint32_t, t);
                continue;
            }
            out[q][i] = __builtin_amdgcn_perm(b, a, 0x07060302u);  // the upper halves
            if (q + 1 < P) {
                a = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) - __builtin_bit_cast(float, a & 0xffff0000u));
                b = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, b) - __builtin_bit_cast(float, b & 0xffff0000u));
            }
        }
}

template <int XT, int G, int RB, int CB, int D, int MODE>
__global__ __launch_bounds__(512) void q4_skinny_kernel(Q4Args p) {
    constexpr bool BF = XT != kXF16;
    constexpr bool F32 = XT == kXF32x2 || XT == kXF32x3;
    constexpr bool EXACT = XT == kXF32x3;                          // codes decoded to code - zero
    constexpr int P = XT == kXF32x3 ? 3 : XT == kXF32x2 ? 2 : 1;  // bfloat16 parts of x
    constexpr int GPU_ = 128 / G;                                  // groups per unit
    constexpr int NC = MODE == kGateUp ? CB / 2 : CB;              // output column blocks
    __shared__ f4 red[8][RB * CB][64];

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, h = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = p.w.K, ku = p.w.ku;
    int e = 0, row0, count;
    if constexpr (MODE == kDense) {
        row0 = blockIdx.y * (16 * RB);
        const int64_t left = p.M - row0;
        count = left < 16 * RB ? (int)left : 16 * RB;
    } else {
        if ((int)blockIdx.y >= *p.ntiles) return;
        const int4 t = p.tiles[blockIdx.y];
        e = t.x, row0 = t.y, count = t.z;
    }
    const int wk = wave & ((1 << p.log_wk) - 1), wn = wave >> p.log_wk, cols = (8 >> p.log_wk) * NC;
    // rows past the last are zeros, not loaded (their results are not stored)
    int64_t xoff[RB];
    bool live[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        live[rb] = rb * 16 + r < count;
        int64_t row = row0 + (live[rb] ? rb * 16 + r : 0);
        if constexpr (MODE == kGateUp) row = p.order[row] / p.topk;
        xoff[rb] = row * K + 8 * h;
    }
    // column blocks past the last repeat it, likewise
    const w4 *cp[CB];
    const uint16_t *sp[CB];
    const uint8_t *zp[CB];
    const bool zeros = p.w.zeros != nullptr;
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        const Q4View &w = MODE == kGateUp && (cb & 1) ? p.w2 : p.w;
        int nb = blockIdx.x * cols + wn * NC + (MODE == kGateUp ? cb >> 1 : cb);
        nb = nb < w.nb ? nb : w.nb - 1;
        const int64_t unit = ((int64_t)e * w.nb + nb) * ku;
        cp[cb] = w.codes + unit * 64;  // the wave's; the lane's part is added at each load
        sp[cb] = w.scales + unit * (16 * GPU_);
        zp[cb] = w.zeros + unit * (16 * GPU_);
    }

    w4 areg[D][RB][F32 ? 8 : 4];
    w4 breg[D][CB];
    uint2 sreg[D][CB];
    uint32_t zreg[D][CB];
    auto load = [&](int st, int u) {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            breg[st][cb] = (cp[cb] + (int64_t)u * 64)[lane];
            const int64_t at = (int64_t)u * (16 * GPU_);
            q4_load_groups<G>(sp[cb] + at, zeros ? zp[cb] + at : nullptr, r, sreg[st][cb], zreg[st][cb]);
        }
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = live[rb] && u * 128 + 32 * j < K;  // K is a multiple of 32
                if constexpr (F32) {
                    const w4 *x = reinterpret_cast<const w4 *>(static_cast<const float *>(p.x) + xoff[rb] + u * 128 + 32 * j);
                    areg[st][rb][2 * j] = in ? x[0] : w4{};
                    areg[st][rb][2 * j + 1] = in ? x[1] : w4{};
                } else {
                    const w4 *x = reinterpret_cast<const w4 *>(static_cast<const uint16_t *>(p.x) + xoff[rb] + u * 128 + 32 * j);
                    areg[st][rb][j] = in ? *x : w4{};
                }
            }
    };
    f4 acc[RB][CB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) acc[rb][cb] = f4{};
    const uint32_t one2 = BF ? 0x3F803F80u : 0x3C003C00u;
    const w4 ones = {one2, one2, one2, one2};
    auto compute = [&](int st) {
        f4 part[RB][CB], sum[RB];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool first = (32 * j) % G == 0, last = (32 * (j + 1)) % G == 0;
            w4 a[RB][P];
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                if constexpr (F32) q4_split<P>(areg[st][rb][2 * j], areg[st][rb][2 * j + 1], a[rb]);
                else a[rb][0] = areg[st][rb][j];
                if constexpr (!EXACT) {
                    if (first) sum[rb] = f4{};
#pragma unroll
                    for (int q = 0; q < P; ++q) sum[rb] = mfma16<BF>(a[rb][q], ones, sum[rb]);
                }
            }
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) {
                w4 b;
                if constexpr (EXACT) b = q4_word_exact(breg[st][cb][j], (float)((zreg[st][cb] >> (8 * (32 * j / G))) & 255u));
                else b = q4_word16<BF>(breg[st][cb][j]);
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
                    if (first) part[rb][cb] = f4{};
#pragma unroll
                    for (int q = 0; q < P; ++q) part[rb][cb] = mfma16<BF>(a[rb][q], b, part[rb][cb]);
                }
            }
            if (last) {
                const int g = 32 * j / G;
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    const float s = half_bits((g & 2 ? sreg[st][cb].y : sreg[st][cb].x) >> (16 * (g & 1)));
                    const float zc = 16.0f + (float)((zreg[st][cb] >> (8 * g)) & 255u);
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[rb][cb][i] += s * (EXACT ? part[rb][cb][i] : part[rb][cb][i] - zc * sum[rb][i]);
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb) q4_here(acc[rb][cb]);  // not behind all products: registers
                }
            }
            if constexpr (RB > 1) __builtin_amdgcn_sched_barrier(0);
        }
    };

    const int step = 1 << p.log_wk, n = (ku - wk + step - 1) >> p.log_wk;  // this wave's units
#pragma unroll
    for (int st = 0; st < D; ++st)
        if (st < n) load(st, wk + step * st);
    for (int t0 = 0; t0 < n; t0 += D) {
#pragma unroll
        for (int st = 0; st < D; ++st) {
            const int t = t0 + st;
            if (t < n) {
                compute(st);
                if (t + D < n) load(st, wk + step * (t + D));
            }
        }
    }

#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) red[wave][rb * CB + cb][lane] = acc[rb][cb];
    __syncthreads();
    // lane l of a tile holds column l%16, rows 4(l/16) .. +3
    auto total = [&](int group, int blk, int row, int col) {
        const int l = (row >> 2) * 16 + col;
        float v = 0.0f;
        for (int q = 0; q < step; ++q) v += red[(group << p.log_wk) + q][blk][l][row & 3];
        return v;
    };
    for (int it = tid; it < RB * cols * 256; it += 512) {
        const int blk = it >> 8, cb = blk % NC, rb = blk / NC % RB, group = blk / (NC * RB);
        const int row = (it & 255) >> 4, col = it & 15;
        const int m = rb * 16 + row, nn = (blockIdx.x * cols + group * NC + cb) * 16 + col;
        if (m >= count || nn >= p.w.N) continue;
        if constexpr (MODE == kDense) {
            float v = total(group, rb * CB + cb, row, col);
            if (!__builtin_isfinite(v)) v = q4_slow_row<XT>(p.x, (int64_t)row0 + m, p.w, 0, nn);
            constexpr int DT = XT == kXF16 ? kF16 : XT == kXBF16 ? kBF16 : kF32;
            store_from_float<DT>(p.y, ((int64_t)row0 + m) * p.w.N + nn, v);
        } else if constexpr (MODE == kGateUp) {
            float g = total(group, rb * CB + 2 * cb, row, col), u = total(group, rb * CB + 2 * cb + 1, row, col);
            if (!__builtin_isfinite(g) || !__builtin_isfinite(u)) {
                const int64_t tok = p.order[row0 + m] / p.topk;
                g = q4_slow_row<XT>(p.x, tok, p.w, e, nn);
                u = q4_slow_row<XT>(p.x, tok, p.w2, e, nn);
            }
            static_cast<float *>(p.y)[((int64_t)row0 + m) * p.w.N + nn] = g / (1.0f + expf(-g)) * u;
        } else {
            float v = total(group, rb * CB + cb, row, col);
            if (!__builtin_isfinite(v)) v = q4_slow_row<XT>(p.x, (int64_t)row0 + m, p.w, e, nn);
            const int slot = p.order[row0 + m];
            static_cast<float *>(p.y)[(int64_t)slot * p.w.N + nn] = p.weights[slot] * v;
        }
    }
}

// The waves per compute unit that a launch wants before it splits a column block's k
// no further.
constexpr int64_t kWavesWanted = 2048;

template <int XT, int G, int RB, int CB, int MODE>
inline hipError_t run_q4_skinny(Q4Args a, int64_t grid_y, hipStream_t s) {
    constexpr int PERX = XT == kXF32x2 || XT == kXF32x3 ? 8 : 4;
    constexpr int REGS = 4 * (RB * PERX + CB);  // registers of one unit in flight
    constexpr int D = REGS <= 48 ? 2 : 1;  // (72 registers twice: 23 f32 rows 20.2 against 16.6 us)
    constexpr int NC = MODE == kGateUp ? CB / 2 : CB;
    const int64_t blocks = (a.w.nb + NC - 1) / NC;
    while (a.log_wk < 3 && (blocks * grid_y << a.log_wk) < kWavesWanted && (2 << a.log_wk) <= a.w.ku) ++a.log_wk;
    const int64_t wn = 8 >> a.log_wk;
    const dim3 grid((unsigned)((blocks + wn - 1) / wn), (unsigned)grid_y);
    q4_skinny_kernel<XT, G, RB, CB, D, MODE><<<grid, dim3(512), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace tq2
