// Products of many rows with a 4-bit weight, on tiles of BM rows by 256 columns.
//
// A workgroup of eight waves; wave w owns two blocks of 16 columns and all BM rows,
// so every code is decoded once per tile.  x comes as f16 planes (q4_prep_kernel) and
// goes through registers into two LDS buffers of 128 k, swizzled so that the 16 rows
// of a fragment read lie on distinct banks; codes and scales go from memory straight
// into the registers of the wave that decodes them, a unit of 128 k ahead.  One barrier
// per unit; while unit u is multiplied, unit u+1 moves into the other buffer and the
// loads of u+2 are sent.
//
// The codes are decoded to code - zero, exact in f16, and each group's sum is scaled in f32:
// acc += scale * part.  Products are exact for f16 x.  bfloat16 rows are
// brought to f16 by a power of two per row (their 8 bits fit; see q4_prep.h), and f32 rows
// to two f16 parts.  silu(g) u of 16-bit rows is held in f16 under a power of two per row and 128
// columns, from its largest value there; the down product brings a row's parts under one power of two.
//
// Bound by the matrix unit and the waits around it: 2048 x 4096 x 4096, G = 128 takes 69-76
// us (0.9-1.0 PFLOP/s; bfloat16 8 more for the planes), with the matrix unit busy 44% of the time,
// LDS 28%, waves at a wait or barrier 35%.  64 experts of 8, 2048 tokens, 2048 x 1024: gate and up 214-224 us (busy
// 40%), down 137-140 (31%; eight units to a tile, and some 5 us for the rows' powers of two).
// Tried without gain: the next unit's codes decoded between this one's products (79.5 against 78 us for
// f16 x), workgroups of four waves, two to a compute unit (94 against 79 us; with G = 32 it gains 9%), halves of
// a tile for an expert's last rows (scratch).
#pragma once

#include <type_traits>

#include "q4.h"

namespace tq2 {

// kTDense: y = x W^T.  kTGateUp: column block 2i is gate's, 2i+1 up's;
// h[p][n] = silu(g) u at sorted place p.  kTDown: part[slot][n] = weight[slot] * sum.
enum Q4TMode { kTDense = 0, kTGateUp = 1, kTDown = 2 };

struct Q4TArgs {
    Q4View w;
    const _Float16 *a;       // [planes][rows][lda]
    int64_t plane, lda;      // elements
    const float *rowscale;   // [rows]: the power of two that each row was divided by (nullptr: 1)
    void *y;
    int64_t M;               // kTDense: rows
    float *part;             // kTDense: the sums of each share of the units (nullptr: one share, y itself)
    int64_t part_stride;
    int split;               // shares
    int tiles_n;
    int topk;
    const int32_t *order;
    const int4 *tiles;
    const int32_t *ntiles;
    const float *weights;
    int16_t *hexp;           // f16 h: q4_h_exp of each place's row and unit of 128 columns, [places][units]
    int64_t ldh;             // kTGateUp, f16 h: row length, whole units of 128 (zeros past N)
    Q4View w2;               // kTGateUp: up
};

__device__ __forceinline__ int q4_lds(int row, int chunk) { return row * 128 + ((chunk ^ (row & 15)) << 3); }

// -(1024 + zero) and -(64 + zero), exact in f16.
struct Q4Zero {
    _Float16 c0, c1;
};
__device__ __forceinline__ Q4Zero q4_zero(uint32_t zero) {
    const _Float16 z = (_Float16)(uint16_t)zero;
    return Q4Zero{(_Float16)-1024.0f - z, (_Float16)-64.0f - z};
}

// code - zero of a word's eight codes: the codes inserted into 1024 (or, four bits
// higher, read as 1024 + 16 code and divided by 16), the zero point taken off; all exact.
__device__ __forceinline__ h8 q4_word_f16(uint32_t w, Q4Zero z, uint32_t magic) {
    constexpr uint32_t m0 = 0x000F000Fu, m1 = 0x00F000F0u;
    const h2 k = {(_Float16)0.0625f, (_Float16)0.0625f}, c0 = {z.c0, z.c0}, c1 = {z.c1, z.c1};
    const uint32_t v = w >> 8;
    const h2 p0 = as_h2((w & m0) | (magic & ~m0)) + c0;
    const h2 p1 = __builtin_elementwise_fma(as_h2((w & m1) | (magic & ~m1)), k, c1);
    const h2 p2 = as_h2((v & m0) | (magic & ~m0)) + c0;
    const h2 p3 = __builtin_elementwise_fma(as_h2((v & m1) | (magic & ~m1)), k, c1);
    return h8{p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
}

// The exponent by which a row with the largest finite value `most` is shifted to bring
// that into [2^14, 2^15) (0 for a row of zeros).
__device__ __forceinline__ int q4_row_shift(float most) {
    int e = 15;
    if (most > 0.0f) (void)__builtin_frexpf(most, &e);  // most in [2^(e-1), 2^e)
    return 15 - e > 126 ? 126 : 15 - e;
}

// The exponent of the power of two by which 128 columns of a row's silu(g) u are divided before they
// are rounded to f16, from the bits of the largest magnitude among them, which comes to [2^14, 2^15).
// (Beside an infinity or NaN finite values only have to stay finite: 114.)
__device__ __forceinline__ int q4_h_exp(uint32_t most) {
    const int e = (int)(most >> 23) - 141;
    return e < -126 ? -126 : e;
}

// The two factors, as halves, that bring such values under a row's power of two, 2^down times as large
// as theirs (down >= 0).  Two, because one would end at 2^-24: what falls below f16 with both is less than
// 2^-39 of the row's largest value.
__device__ __forceinline__ uint32_t q4_h_factors(int down) {
    down = down < 48 ? down : 48;
    const int half = down >> 1;
    const h2 f = {(_Float16)__builtin_ldexpf(1.0f, -half), (_Float16)__builtin_ldexpf(1.0f, half - down)};
    return __builtin_bit_cast(uint32_t, f);
}
__device__ __forceinline__ w4 q4_h_lower(w4 v, uint32_t factors) {
    const h2 f = as_h2(factors), a = {f.x, f.x}, b = {f.y, f.y};
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = __builtin_bit_cast(uint32_t, as_h2(v[q]) * a * b);
    return v;
}

// silu(g) u for a consumer that rounds to f16: e^-g and the quotient from the hardware's exp2 and
// reciprocal, relative error below 2^-17 (of it |g| 2^-24 from the rounded exponent).
__device__ __forceinline__ float q4_silu_f16(float g, float u) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f)) * u;
}

template <int BM, int G, int P, int MODE, int DT>
__global__ __launch_bounds__(512) void q4_tiled_kernel(Q4TArgs p) {
    constexpr int RB = BM / 16, GPU_ = 128 / G, NCB = 2;
    constexpr int FRAG = P == 1;                  // fragments are read a row block ahead where registers allow
    constexpr int PPT = BM * 16 / 512;  // 16-byte pieces of a plane's tile per thread
    __shared__ __attribute__((aligned(16))) _Float16 As[2][P][BM * 128];
    constexpr bool H16 = P == 1 && MODE != kTDense;   // h in f16 under powers of two
    __shared__ __attribute__((aligned(16))) float rs[BM], slot_weight[MODE == kTDown ? BM : 4];
    __shared__ __attribute__((aligned(16))) int slots[MODE == kTDown ? BM : 4];
    // kTGateUp: bits of the largest magnitude of the row's h in this tile
    __shared__ __attribute__((aligned(16))) int hmost[H16 && MODE == kTGateUp ? BM : 4];
    constexpr int TU = 64;  // kTDown: units whose factors are at hand
    __shared__ uint32_t factors[H16 && MODE == kTDown ? TU * BM : 1];

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, h = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ku = p.w.ku;
    // kTDense: the units are dealt to gridDim.y workgroups
    const int u_begin = MODE == kTDense ? (int)((int64_t)ku * blockIdx.y / gridDim.y) : 0;
    const int u_end = MODE == kTDense ? (int)((int64_t)ku * (blockIdx.y + 1) / gridDim.y) : ku;
    const uint32_t magic = f16_magic();

    // Workgroups go round the 8 XCDs: give each XCD a run of neighbouring tiles, N first.
    int tile = blockIdx.x;
    const int tiles = gridDim.x;
    if ((tiles & 7) == 0) tile = (tile & 7) * (tiles >> 3) + (tile >> 3);
    const int tn = tile % p.tiles_n, tm = tile / p.tiles_n;
    int e = 0, count;
    int64_t row0;
    if constexpr (MODE == kTDense) {
        row0 = (int64_t)tm * BM;
        if (row0 >= p.M) return;  // the grid is whole runs of tiles; the whole workgroup
        count = p.M - row0 < BM ? (int)(p.M - row0) : BM;
    } else {
        if (tm >= *p.ntiles) return;  // the whole workgroup
        const int4 t = p.tiles[tm];
        e = t.x, row0 = t.y, count = t.z;
    }
    auto source = [&](int row) -> int64_t {  // row of A; rows past the last repeat it
        const int64_t at = row0 + (row < count ? row : count - 1);
        return MODE == kTGateUp ? (int64_t)(p.order[at] / p.topk) : at;
    };
    if (tid < BM) {
        const int64_t s = source(tid);
        if constexpr (!(H16 && MODE == kTDown)) rs[tid] = p.rowscale ? p.rowscale[s] : 1.0f;
        if constexpr (MODE == kTDown) {
            const int slot = p.order[s];
            slots[tid] = slot;
            slot_weight[tid] = p.weights[slot];  // (its product with the row's power of two may leave f32's range)
        }
        if constexpr (H16 && MODE == kTGateUp) hmost[tid] = 0;
    }
    // A row's power of two is the largest of its units'; 512/BM neighbouring threads serve a row.
    constexpr int LANES = 512 / BM;
    auto fill_factors = [&](int u0, int row_exp) {
        const int16_t *ex = p.hexp + source(tid / LANES) * ku;
        for (int u = u0 + tid % LANES; u < ku && u < u0 + TU; u += LANES)
            factors[(u - u0) * BM + tid / LANES] = q4_h_factors(row_exp - ex[u]);
    };
    const _Float16 *ap[PPT];
    int al[PPT];
#pragma unroll
    for (int c = 0; c < PPT; ++c) {
        const int piece = tid + c * 512, row = piece >> 4, chunk = piece & 15;
        ap[c] = p.a + source(row) * p.lda + chunk * 8;
        al[c] = q4_lds(row, chunk);
    }
    const w4 *cp[NCB];
    const uint16_t *sp[NCB];
    const uint8_t *zp[NCB];
    const bool zeros = p.w.zeros != nullptr;
    int nb[NCB];
#pragma unroll
    for (int cb = 0; cb < NCB; ++cb) {
        const Q4View &w = MODE == kTGateUp && cb ? p.w2 : p.w;
        nb[cb] = MODE == kTGateUp ? tn * 8 + wave : tn * 16 + wave * 2 + cb;
        const int at = nb[cb] < w.nb ? nb[cb] : w.nb - 1;  // past the last: its results are not stored
        const int64_t unit = ((int64_t)e * w.nb + at) * ku;
        cp[cb] = w.codes + unit * 64;  // the wave's; the lane's part is added at each load
        sp[cb] = w.scales + unit * (16 * GPU_);
        zp[cb] = w.zeros + unit * (16 * GPU_);
    }
    w4 areg[P][PPT];
    auto load_a = [&](int u) {
#pragma unroll
        for (int q = 0; q < P; ++q)
#pragma unroll
            for (int c = 0; c < PPT; ++c) areg[q][c] = *reinterpret_cast<const w4 *>(ap[c] + q * p.plane + (int64_t)u * 128);
    };
    auto store_a = [&](int buf, int u) {  // unit u
        if constexpr (H16 && MODE == kTDown)
#pragma unroll
            for (int c = 0; c < PPT; ++c)
                areg[0][c] = q4_h_lower(areg[0][c], factors[(u % TU) * BM + (tid >> 4) + 32 * c]);
#pragma unroll
        for (int q = 0; q < P; ++q)
#pragma unroll
            for (int c = 0; c < PPT; ++c) *reinterpret_cast<w4 *>(&As[buf][q][al[c]]) = areg[q][c];
    };
    w4 breg[2][NCB];
    uint2 sreg[2][NCB];
    uint32_t zreg[2][NCB];
    auto load_b = [&](int st, int u) {
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb) {
            breg[st][cb] = (cp[cb] + (int64_t)u * 64)[lane];
            const int64_t at = (int64_t)u * (16 * GPU_);
            q4_load_groups<G>(sp[cb] + at, zeros ? zp[cb] + at : nullptr, r, sreg[st][cb], zreg[st][cb]);
        }
    };

    f4 acc[RB][NCB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb) acc[rb][cb] = f4{};
    h8 b[NCB][4];
    auto decode = [&](int st) {
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                b[cb][j] = q4_word_f16(breg[st][cb][j], q4_zero((zreg[st][cb] >> (8 * (32 * j / G))) & 255u), magic);
    };
    // The two waves of a SIMD should not decode at the same time.  A wave at its products goes first
    // (14336 x 4096, G = 32, 1024 rows 170 -> 160 us; 64 experts, 128 tokens 128 -> 124); with two planes
    // half of the waves also decode before the barrier instead of after it (f32, 2048 rows, G = 32
    // 532 -> 503 us; one plane: no gain).
    const bool late = P == 2 && wave >= 4;
    auto compute = [&](int buf, int st, auto &&hook) {
        if (!late) decode(st);
        __builtin_amdgcn_s_setprio(1);
        h8 a[1 + FRAG][P][4];
        auto fragments = [&](int rb) {
#pragma unroll
            for (int q = 0; q < P; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    a[rb & FRAG][q][j] = *reinterpret_cast<const h8 *>(&As[buf][q][q4_lds(rb * 16 + r, 4 * j + h)]);
        };
        // Step t: column block t % NCB of row block t / NCB.  The previous step's parts are scaled
        // while this one's products run, and no later: left free, the compiler puts all scaling
        // behind all products, whose parts then go to scratch memory (G = 32, 1024 x 14336 x 4096: 1337
        // against 170 us then; G = 64, 2048 x 4096 x 4096: 132 against 74).  One part a step fits the registers
        // as it is (G = 128: 79 us, held in place 84).
        f4 part[2][GPU_];
        auto scale = [&](int t) {
            const int rb = t / NCB, cb = t % NCB;
#pragma unroll
            for (int g = 0; g < GPU_; ++g) {
                const float s = half_bits((g & 2 ? sreg[st][cb].y : sreg[st][cb].x) >> (16 * (g & 1)));
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[rb][cb][i] += s * part[t & 1][g][i];
            }
            if constexpr (GPU_ > 1 || P > 1) q4_here(acc[rb][cb]);
        };
        if (FRAG) fragments(0);
#pragma unroll
        for (int t = 0; t < RB * NCB; ++t) {
            const int rb = t / NCB, cb = t % NCB;
            if (cb == 0 && rb + FRAG < RB) fragments(rb + FRAG);
#pragma unroll
            for (int g = 0; g < GPU_; ++g) {
                part[t & 1][g] = f4{};
#pragma unroll
                for (int q = P - 1; q >= 0; --q)
#pragma unroll
                    for (int j = g * G / 32; j < (g + 1) * G / 32; ++j)
                        part[t & 1][g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[rb & FRAG][q][j], b[cb][j], part[t & 1][g], 0, 0, 0);
            }
            if (t > 0) scale(t - 1);
            if (t == NCB) hook();
        }
        scale(RB * NCB - 1);
        __builtin_amdgcn_s_setprio(0);
        if (late) decode(st ^ 1);
    };

    auto last = [&](int u) { return u < u_end ? u : u_end - 1; };
    load_a(u_begin);
    load_b(0, u_begin);
    if constexpr (H16 && MODE == kTDown) {  // behind the first loads, on their way
        const int16_t *ex = p.hexp + source(tid / LANES) * ku;
        int row_exp = -126;
        for (int u = tid % LANES; u < ku; u += LANES) row_exp = ex[u] > row_exp ? ex[u] : row_exp;
        for (int o = 1; o < LANES; o <<= 1) {
            const int b = __shfl_xor(row_exp, o);
            row_exp = b > row_exp ? b : row_exp;
        }
        if (tid % LANES == 0) rs[tid / LANES] = __builtin_ldexpf(1.0f, row_exp);
        fill_factors(0, row_exp);
        __syncthreads();
    }
    load_b(1, last(u_begin + 1));
    store_a(0, u_begin);
    load_a(last(u_begin + 1));
    if (late) decode(0);
    __syncthreads();
    for (int u0 = u_begin; u0 < u_end; u0 += 2) {
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const int u = u0 + st;
            if (u < u_end) {
                compute(st, st, [&] {
                    store_a(st ^ 1, u + 1);
                    load_a(last(u + 2));
                });
                load_b(st, last(u + 2));
                __syncthreads();
                if constexpr (H16 && MODE == kTDown)
                    if ((u + 2) % TU == 0) {  // the next unit that is stored is the first of others
                        const float scale = rs[tid / LANES];
                        fill_factors(u + 2, (int)(__builtin_bit_cast(uint32_t, scale) >> 23) - 127);
                        __syncthreads();
                    }
            }
        }
    }

    if constexpr (MODE == kTGateUp && H16) {  // a tile covers a whole unit of h
        const int n = nb[0] * 16 + r;
        uint32_t most[RB * 4];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
            for (int i = 0; i < 4; ++i) most[rb * 4 + i] = 0;
            if (rb * 16 >= count) continue;  // the whole wave
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float scale = rs[rb * 16 + 4 * h + i];
                const float v = n < p.w.N ? q4_silu_f16(acc[rb][0][i] * scale, acc[rb][1][i] * scale) : 0.0f;
                acc[rb][0][i] = v;
                most[rb * 4 + i] = __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;  // (of the vector's element it would be element 0's)
            }
        }
        // the largest of each row: every exchange halves the rows that a lane keeps
        int first = 0;  // its first row, counted as rb * 4 + i
        auto halve = [&](auto exchange, int bit, int keep) {
            const bool upper = (r & bit) != 0;
            first += upper ? keep : 0;
#pragma unroll
            for (int j = 0; j < keep; ++j) {
                const uint32_t mine = upper ? most[j + keep] : most[j], other = upper ? most[j] : most[j + keep];
                const uint32_t got = exchange(other);
                most[j] = mine > got ? mine : got;
            }
        };
        auto swapped = [](auto ctrl) {
            return [](uint32_t v) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, decltype(ctrl)::value, 0xF, 0xF, false); };
        };
        halve(swapped(std::integral_constant<int, 0xB1>{}), 1, RB * 2);   // lane ^ 1
        halve(swapped(std::integral_constant<int, 0x4E>{}), 2, RB);       // lane ^ 2
        halve(swapped(std::integral_constant<int, 0x124>{}), 4, RB / 2);  // lane - 4 of the sixteen
        halve(swapped(std::integral_constant<int, 0x128>{}), 8, RB / 4);  // lane ^ 8
#pragma unroll
        for (int j = 0; j < RB / 4; ++j) {
            const int at = first + j;
            atomicMax(&hmost[(at >> 2) * 16 + 4 * h + (at & 3)], (int)most[j]);
        }
        __syncthreads();
        if (tid < count) p.hexp[(row0 + tid) * p.tiles_n + tn] = (int16_t)q4_h_exp(hmost[tid]);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            if (rb * 16 >= count) break;
            const int4 bits = *reinterpret_cast<const int4 *>(&hmost[rb * 16 + 4 * h]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = rb * 16 + 4 * h + i;
                if (m >= count) continue;
                const int e = q4_h_exp(i == 0 ? bits.x : i == 1 ? bits.y : i == 2 ? bits.z : bits.w);
                static_cast<_Float16 *>(p.y)[(row0 + m) * p.ldh + n] = (_Float16)__builtin_ldexpf(acc[rb][0][i], -e);
            }
        }
        return;
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        if constexpr (MODE == kTGateUp) {
            const int n = nb[0] * 16 + r;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = rb * 16 + 4 * h + i;
                if (m >= count || n >= p.w.N) continue;
                const float g = acc[rb][0][i] * rs[m], u = acc[rb][1][i] * rs[m];
                static_cast<float *>(p.y)[(row0 + m) * p.w.N + n] = g / (1.0f + expf(-g)) * u;
            }
        } else if constexpr (MODE == kTDown) {
            const int m = rb * 16 + 4 * h;
            const f4 scale = *reinterpret_cast<const f4 *>(&rs[m]), weight = *reinterpret_cast<const f4 *>(&slot_weight[m]);
            const int4 s4 = *reinterpret_cast<const int4 *>(&slots[m]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (m + i >= count) continue;
                const int slot = i == 0 ? s4.x : i == 1 ? s4.y : i == 2 ? s4.z : s4.w;
                float *out = static_cast<float *>(p.y) + (int64_t)slot * p.w.N;
#pragma unroll
                for (int cb = 0; cb < NCB; ++cb) {
                    const int n = nb[cb] * 16 + r;
                    if (n < p.w.N) out[n] = weight[i] * (acc[rb][cb][i] * scale[i]);
                }
            }
        } else {
#pragma unroll
            for (int cb = 0; cb < NCB; ++cb) {
                const int n = nb[cb] * 16 + r;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = rb * 16 + 4 * h + i;
                    if (m >= count || n >= p.w.N) continue;
                    const float v = acc[rb][cb][i] * rs[m];
                    const int64_t at = (row0 + m) * p.w.N + n;
                    if (p.part) p.part[blockIdx.y * p.part_stride + at] = v;
                    else store_from_float<DT>(p.y, at, v);
                }
            }
        }
    }
}

template <int BM, int G, int P, int MODE, int DT>
inline hipError_t run_q4_tiled(Q4TArgs a, int64_t tiles_m, hipStream_t s) {
    a.tiles_n = MODE == kTGateUp ? (a.w.nb + 7) / 8 : (a.w.nb + 15) / 16;
    const int64_t grid = (tiles_m * a.tiles_n + 7) / 8 * 8;
    const dim3 blocks((unsigned)grid, MODE == kTDense ? (unsigned)a.split : 1);
    q4_tiled_kernel<BM, G, P, MODE, DT><<<blocks, dim3(512), 0, s>>>(a);
    return hipGetLastError();
}

// x as f16 planes (see q4_prep.h).
struct Q4Prep {
    const void *x;
    int64_t row0, rows;      // row0: of the launch
    int K;
    int64_t lda, plane;      // of the planes (elements)
    _Float16 *out;
    float *rowscale;
};
hipError_t launch_q4_prep(Q4Prep p, int dtype, hipStream_t s);
// Whether x is read as it is: f16 rows of whole units.
inline bool q4_plain_x(int64_t K, int dtype) { return dtype == kF16 && K % 128 == 0; }
inline int q4_planes(int dtype) { return dtype == kF32 ? 2 : 1; }
hipError_t launch_q4_tiled_dense(const Q4TArgs &a, int dtype, int bm, hipStream_t s);
hipError_t launch_q4_join(const float *part, int64_t stride, int split, void *y, int64_t n, int dtype, hipStream_t s);
hipError_t launch_q4_tiled_gate_up(const Q4TArgs &a, int planes, int bm, int64_t tiles, hipStream_t s);
hipError_t launch_q4_tiled_down(const Q4TArgs &a, int planes, int bm, int64_t tiles, hipStream_t s);

}  // namespace tq2
