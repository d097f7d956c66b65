// Experts' products with few rows each: a workgroup finds its expert's slots by itself.
//
// Workgroup (x, e, z) of eight waves looks through the T*k chosen experts for e, and takes
// e's slots 16 rows at a time, the z-th of them in turn: it brings their rows to LDS as f16
// planes (f16 rows as they are; bfloat16 and f32 rows, whole in a wave's registers, under a
// power of two per row as q4_prep.h makes them), and its waves multiply them with CB
// column blocks each.
// WK waves share a column block and take its units in turn; their sums are added in wave order.
// Only codes and scales wait in registers, D units ahead: these products wait for
// memory.  Codes are decoded to code - zero, exact in f16, and each group's sum is scaled in f32.
// 33 tokens of 32 experts, 4 each, 1024 x 1536, f16: gate and up 15-17 us (3.2-3.6 TB/s of codes and
// scales), down 12 (2.3 TB/s); a plan, tiles and f32 rows through the skinny kernel took 46 in all.
// 128 registers let two workgroups share a compute unit, for up to 84 bytes a lane in scratch memory.
#pragma once

#include "q4_tiled.h"

namespace tq2 {

// kGroupGateUp: h[slot][n] = silu(g) u (f32).  kGroupDown: part[slot][n] = weight * (h W^T) (f32).
enum Q4GroupMode { kGroupGateUp = 0, kGroupDown = 1 };
constexpr int kGroupMaxK = 2048;      // a row in a wave's registers: 32 values a lane
constexpr int kGroupMaxSlots = 2048;

struct Q4GroupArgs {
    Q4View w;                // kGroupGateUp: gate
    const void *x;           // kGroupGateUp: x [T][K]; kGroupDown: h [slots][K], f32
    float *y;
    const int32_t *idx;
    const float *weights;
    int slots, topk, log_wk;
    Q4View w2;               // kGroupGateUp: up
};

template <int DT, int P, int G, int CB, int D, int MODE>
__global__ __launch_bounds__(512, 4) void q4_group_kernel(Q4GroupArgs p) {
    constexpr int GPU_ = 128 / G, NC = MODE == kGroupGateUp ? CB / 2 : CB, RB = 1, ROWS = 16 * RB;
    extern __shared__ __attribute__((aligned(16))) _Float16 xs[];  // [P][ROWS][128 ku]
    __shared__ f4 red[8][RB * CB][64];
    __shared__ float rs[ROWS];
    __shared__ uint16_t list[kGroupMaxSlots];  // this expert's slots
    __shared__ int wcount[8];

    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, h = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int K = p.w.K, ku = p.w.ku, kp = ku * 128, e = blockIdx.y;
    const uint32_t magic = f16_magic();

    const int step = 1 << p.log_wk, wk = wave & (step - 1), wn = wave >> p.log_wk, cols = (8 >> p.log_wk) * NC;
    const w4 *cp[CB];
    const uint16_t *sp[CB];
    const uint8_t *zp[CB];
    const bool zeros = p.w.zeros != nullptr;
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        const Q4View &w = MODE == kGroupGateUp && (cb & 1) ? p.w2 : p.w;
        int nb = blockIdx.x * cols + wn * NC + (MODE == kGroupGateUp ? cb >> 1 : cb);
        nb = nb < w.nb ? nb : w.nb - 1;  // past the last: not stored
        const int64_t unit = ((int64_t)e * w.nb + nb) * ku;
        cp[cb] = w.codes + unit * 64;  // the wave's; the lane's part is added at each load
        sp[cb] = w.scales + unit * (16 * GPU_);
        zp[cb] = w.zeros + unit * (16 * GPU_);
    }
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
    };
    const int n = (ku - wk + step - 1) >> p.log_wk;  // this wave's units: wk, wk + step, ...

    // the first units' codes are on their way while the slots are found
    auto first_units = [&] {
#pragma unroll
        for (int st = 0; st < D; ++st)
            if (st < n) load(st, wk + step * st);
    };
    if (blockIdx.z == 0) first_units();

    // the expert's slots, in order
    int count = 0;
    for (int s0 = 0; s0 < p.slots; s0 += 512) {
        const bool mine = s0 + tid < p.slots && p.idx[s0 + tid] == e;
        const uint64_t who = __ballot(mine);
        if (lane == 0) wcount[wave] = __popcll(who);
        __syncthreads();
        int at = count;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q < wave) at += wcount[q];
            count += wcount[q];
        }
        if (mine) list[at + __popcll(who & ((1ull << lane) - 1))] = (uint16_t)(s0 + tid);
        __syncthreads();
    }
    if (count <= (int)blockIdx.z * ROWS) return;  // the whole workgroup

    for (int c0 = blockIdx.z * ROWS; c0 < count; c0 += ROWS * gridDim.z) {
        const int rows = count - c0 < ROWS ? count - c0 : ROWS;
        if (c0 > 0) first_units();  // (the first sixteen rows': above)

        // every wave brings its share of the rows to LDS; those past the last hold zeros
#pragma unroll 1
        for (int row = wave; row < ROWS; row += 8) {
            constexpr int V = DT == kF32 ? 4 : 8, C = kGroupMaxK / 64 / V;  // values and pieces of a lane
            typedef _Float16 hv __attribute__((ext_vector_type(V)));
            const bool live = row < rows;
            const int64_t src = !live ? 0 : MODE == kGroupGateUp ? list[c0 + row] / p.topk : list[c0 + row];
            w4 raw[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = (lane + 64 * c) * V;
                raw[c] = w4{};
                if (live && k < K) {  // K is a multiple of 32
                    if constexpr (DT == kF32) raw[c] = *reinterpret_cast<const w4 *>(static_cast<const float *>(p.x) + src * K + k);
                    else raw[c] = *reinterpret_cast<const w4 *>(static_cast<const uint16_t *>(p.x) + src * K + k);
                }
            }
            int shift = 0;
            auto value = [&](int c, int q) -> float {
                if constexpr (DT == kF32) {
                    const uint32_t v = raw[c][q];  // (a bit cast of the element itself would take element 0)
                    return __builtin_bit_cast(float, v);
                }
                return __builtin_bit_cast(float, q & 1 ? raw[c][q >> 1] & 0xffff0000u : raw[c][q >> 1] << 16);
            };
            if constexpr (DT != kF16) {
                float most = 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        const float a = __builtin_fabsf(value(c, q));
                        most = a > most && a < __builtin_inff() ? a : most;
                    }
                for (int o = 1; o < 64; o <<= 1) most = fmaxf(most, __shfl_xor(most, o));
                shift = q4_row_shift(most);
            }
            if (lane == 0) rs[row] = __builtin_ldexpf(1.0f, -shift);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int i = lane + 64 * c, k = i * V;
                if (k >= kp) continue;
                const int chunk = k >> 3;
                const int at = row * kp + (((chunk & ~15) | ((chunk ^ row) & 15)) << 3) + (k & 7);
                if constexpr (DT == kF16) {
                    *reinterpret_cast<w4 *>(&xs[at]) = raw[c];
                } else {
                    hv a, b;
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        const float x = __builtin_ldexpf(value(c, q), shift);
                        a[q] = (_Float16)x;
                        if constexpr (P == 2) b[q] = __builtin_isfinite(x) ? (_Float16)(x - (float)a[q]) : (_Float16)0.0f;
                    }
                    *reinterpret_cast<hv *>(&xs[at]) = a;
                    if constexpr (P == 2) *reinterpret_cast<hv *>(&xs[ROWS * kp + at]) = b;
                }
            }
        }
        __syncthreads();

        f4 acc[RB][CB];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) acc[rb][cb] = f4{};
        auto compute = [&](int st, int u) {
            f4 part[RB][CB];
            Q4Zero zero[CB];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool first = (32 * j) % G == 0, last = (32 * (j + 1)) % G == 0;
                const int g = 32 * j / G;
                h8 a[RB][P];
#pragma unroll
                for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                    for (int q = 0; q < P; ++q)
                        a[rb][q] = *reinterpret_cast<const h8 *>(
                            &xs[(q * ROWS + rb * 16 + r) * kp + u * 128 + (((4 * j + h) ^ r) << 3)]);
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) {
                    if (first) zero[cb] = q4_zero((zreg[st][cb] >> (8 * g)) & 255u);
                    const h8 b = q4_word_f16(breg[st][cb][j], zero[cb], magic);
                    const float s = half_bits((g & 2 ? sreg[st][cb].y : sreg[st][cb].x) >> (16 * (g & 1)));
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb) {
                        if (first) part[rb][cb] = f4{};
#pragma unroll
                        for (int q = P - 1; q >= 0; --q)
                            part[rb][cb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[rb][q], b, part[rb][cb], 0, 0, 0);
                        if (last) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[rb][cb][i] += s * part[rb][cb][i];
                            q4_here(acc[rb][cb]);
                        }
                    }
                }
            }
        };
        for (int t0 = 0; t0 < n; t0 += D) {
#pragma unroll
            for (int st = 0; st < D; ++st) {
                const int t = t0 + st;
                if (t < n) {
                    compute(st, wk + step * t);
                    if (t + D < n) load(st, wk + step * (t + D));
                    __builtin_amdgcn_sched_barrier(0);  // one unit's decode at a time: registers
                }
            }
        }
        if (step > 1) {  // wave 0 of each column block adds the others' sums
            if (wk) {
#pragma unroll
                for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) red[wave][rb * CB + cb][lane] = acc[rb][cb];
            }
            __syncthreads();
            if (wk == 0)
                for (int q = 1; q < step; ++q)
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                        for (int cb = 0; cb < CB; ++cb) acc[rb][cb] += red[wave + q][rb * CB + cb][lane];
        }
        if (wk == 0) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = rb * 16 + 4 * h + i;
                    if (row >= rows) continue;
                    const int slot = list[c0 + row];
                    const float scale = rs[row];
#pragma unroll
                    for (int cb = 0; cb < NC; ++cb) {
                        const int nn = (blockIdx.x * cols + wn * NC + cb) * 16 + r;
                        if (nn >= p.w.N) continue;
                        float v;
                        if constexpr (MODE == kGroupGateUp) {
                            const float g = acc[rb][2 * cb][i] * scale, u = acc[rb][2 * cb + 1][i] * scale;
                            v = g / (1.0f + expf(-g)) * u;
                        } else {
                            v = p.weights[slot] * (acc[rb][cb][i] * scale);
                        }
                        p.y[(int64_t)slot * p.w.N + nn] = v;
                    }
                }
        }
        __syncthreads();  // the rows' LDS and the sums' are free again
    }
}

inline size_t q4_group_lds(int64_t K, int planes, int rows) { return (size_t)planes * rows * ((K + 127) / 128 * 128) * 2; }
constexpr size_t kGroupLds = 128 * 1024;

template <int DT, int P, int G, int CB, int D, int MODE>
inline hipError_t run_q4_group(Q4GroupArgs a, hipStream_t s) {
    constexpr int NC = MODE == kGroupGateUp ? CB / 2 : CB;
    const int64_t blocks = (a.w.nb + NC - 1) / NC;
    // waves share a column block until there are eight for each compute unit
    const int64_t busy = a.w.E < a.slots ? a.w.E : a.slots;
    while (a.log_wk < 3 && (blocks * busy << a.log_wk) < 2048 && (2 << a.log_wk) <= a.w.ku) ++a.log_wk;
    const int64_t wn = 8 >> a.log_wk;
    // popular experts' blocks of 16 rows go side by side (64 tokens of 32 experts, 4 each: 55 -> 42 us;
    // 24 of 64, 8 each, the few blocks past the first do not pay for the workgroups: 77 -> 83)
    const unsigned z = a.slots > 4 * a.w.E ? 3 : 1;
    q4_group_kernel<DT, P, G, CB, D, MODE>
        <<<dim3((unsigned)((blocks + wn - 1) / wn), (unsigned)a.w.E, z), dim3(512), q4_group_lds(a.w.K, P, 16), s>>>(a);
    return hipGetLastError();
}

hipError_t launch_q4_group_gate_up(const Q4GroupArgs &a, int dtype, hipStream_t s);
hipError_t launch_q4_group_down(const Q4GroupArgs &a, int planes, hipStream_t s);

}  // namespace tq2
