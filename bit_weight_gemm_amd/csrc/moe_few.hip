// A few tokens through a mixture's experts in one launch, from the router's logits: y[t] = residual[t] +
// sum_j w_j down_e(silu(gate_e n_t) * (up_e n_t)), for weights in groups of 128.
//
// Tasks: the slots' gate and up products (32 columns of one slot each), then the down products (16 columns of one token each),
// dealt to at most 512 workgroups in turn.  Each wave chooses some tokens' experts from the logits first (against a
// launch of its own).  A down task sends the loads of its first codes and then reads silu(g) u, which may not be there yet:
// the launch before has filled it with a pattern that no value has, and who reads the pattern reads again.  So nobody counts
// and nothing is fenced.  (384 tickets and 256 counts at one address took one token 34 us, fences at device scope, which write back
// and empty a whole L2 each, 52.)
//
// Every wait ends.  Gate and up tasks wait for nobody, and a workgroup has its own behind it when it waits; the hardware starts workgroups
// in order; but should a down task have looked `patience` times for a value, because the workgroup that has it is not
// running, it gives up, forms its token's silu(g) u itself (the same values at the same places) and begins again.
//
// One token of 8 of 64 experts, 2048 x 1024, bf16: 16.0 us, the least of 30 15.4 (inputs in turn).  The choice 2.5, the codes of all
// products (25 MB, 3.5 TB/s) 7, silu(g) u from one workgroup to the next 2, the down products 3.  As three launches 14 us of kernels and
// their gaps: the same, for two launches' time of the host.  The 128 registers that two workgroups to a compute unit leave a lane
// do not hold all: 20 to 36 bytes of a lane lie in scratch.
// Products, decode, correction and the treatment of infinities are q4_row.h's.
#include "moe_layer.h"
#include "moe_route.h"
#include "q4_epilogue.h"
#include "q4_row.h"

namespace tq2 {

namespace {

constexpr int kFewWaves = 8, kFewSlots = 64;
static_assert(kFewGroup == 128, "a unit has one group");

// Bits of an element of h that is not written yet: a NaN that no part of one is stored as.
constexpr uint16_t kNoH = 0xffff;
__device__ __forceinline__ bool has_none(uint64_t four) {  // one of four halves is kNoH: its complement has a zero half
    return ((~four - 0x0001000100010001ull) & four & 0x8000800080008000ull) != 0;
}

// The argument block is read line by line, each from far: a call has three lines of 64 bytes, and asks for all of them at once.
struct FewWeight {
    const w4 *codes;
    const uint16_t *scales;
    const uint8_t *zeros;
};
struct FewCall {
    FewWeight gate, up, down;
    const void *n, *residual;
    uint16_t *h;             // [T k][PH][ldh], whole units of 128
    void *y;
    const float *logits, *bias;
    int32_t *idx;
    float *weights;
    int E, d, f, T, k, gx, dx;  // gx, dx: tasks of a slot, and of a token's down products
    int patience, room;      // room: halves of LDS before the sums
    int groups, keep, per_group, log_lanes;
    int flags;               // kFew...
};
static_assert(sizeof(FewCall) <= 192, "three lines");
enum { kFewSigmoid = 1, kFewRenorm = 2, kFewTopTwo = 4, kFewOne = 8 };  // kFewOne: a lane of the router has one expert at most

__device__ __forceinline__ Q4View few_view(const FewWeight &w, int E, int N, int K) {
    Q4View v{};
    v.codes = w.codes, v.scales = w.scales, v.zeros = w.zeros, v.E = E, v.N = N, v.K = K, v.G = kFewGroup;
    v.nb = (N + 15) >> 4, v.ku = (K + 127) >> 7;
    return v;
}

// A column block's units, one after another.
struct Units {
    const w4 *codes;
    const uint16_t *scales;
    const uint8_t *zeros;
    __device__ Units(const FewWeight &w, int64_t unit) {
        codes = w.codes + unit * 64, scales = w.scales + unit * 16, zeros = w.zeros ? w.zeros + unit * 16 : nullptr;
    }
    __device__ __forceinline__ void load(int u, int lane, w4 &b, uint2 &s, uint32_t &z) const {
        b = (codes + u * 64)[lane];
        q4_load_groups<kFewGroup>(scales + u * 16, zeros ? zeros + u * 16 : nullptr, lane & 15, s, z);
    }
};

// acc[cb] += weight times a unit of CB column blocks times a row.  The row's P parts are rows of the matrix instruction (its
// other rows repeat the last part): one instruction for all of them, where one each took 16 and with the sums of x by another
// against ones 32 to a unit.  xs: the lane's part, from its first column on; sums: of x over the unit, the parts' pitch apart.
template <int XT, int CB>
__device__ __forceinline__ void few_unit(const uint16_t *xs, const float *sums, int pitch, const w4 *b, const uint2 *s, const uint32_t *z,
                                         float weight, float (&acc)[CB]) {
    constexpr bool BF = XT != kXF16, EXACT = XT == kXF32x3;
    constexpr int P = XT == kXF32x3 ? 3 : XT == kXF32x2 ? 2 : 1;
    f4 part[CB] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const w4 a = *reinterpret_cast<const w4 *>(xs + 32 * j);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            w4 w;
            if constexpr (EXACT) w = q4_word_exact(b[cb][j], (float)(z[cb] & 255u));
            else w = q4_word16<BF>(b[cb][j]);
            part[cb] = mfma16<BF>(a, w, part[cb]);
        }
    }
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        float v = part[cb][0];
#pragma unroll
        for (int q = 1; q < P; ++q) v += part[cb][q];
        if constexpr (!EXACT) {
            float sum = sums[0];
#pragma unroll
            for (int q = 1; q < P; ++q) sum += sums[q * pitch];
            v -= (16.0f + (float)(z[cb] & 255u)) * sum;
        }
        acc[cb] += weight * half_bits(s[cb].x) * v;
    }
}

// Sum of the eight values of a piece, over the sixteen lanes that hold its unit's pieces; for those of f16 or bfloat16.
template <bool BF>
__device__ __forceinline__ float unit_sum(w4 v) {
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (BF) s += __builtin_bit_cast(float, v[q] << 16) + __builtin_bit_cast(float, v[q] & 0xffff0000u);
        else s += half_bits(v[q]) + half_bits(v[q] >> 16);
    }
    s += dpp<0xB1>(s), s += dpp<0x4E>(s);    // lane ^ 1, lane ^ 2
    s += dpp<0x141>(s), s += dpp<0x140>(s);  // mirrored in eight lanes, in sixteen
    return s;
}

// h of 32 columns of a slot with expert e (below 0: dropped, h is 0).
template <int XT, int PH>
__device__ __forceinline__ void up_task(const FewCall &p, int slot, int t, int bx, int e, uint16_t *xs, float *sums, float (*red)[64]) {
    constexpr bool F32 = XT == kXF32x3;
    constexpr int P = F32 ? 3 : 1, CB = 4, D = 2, WAVES = kFewWaves;
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ku = (p.d + 127) >> 7, kh = (p.f + 127) >> 7, nb = (p.f + 15) >> 4;
    const int col = bx * 32 + tid;
    uint16_t *out = p.h + (int64_t)slot * PH * kh * 128 + col;
    if (e < 0) {
        if (tid < 32 && col < p.f)
#pragma unroll
            for (int q = 0; q < PH; ++q) __hip_atomic_store(out + q * kh * 128, (uint16_t)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return;
    }
    const int64_t u0 = ((int64_t)e * nb + 2 * bx) * ku, u1 = u0 + (2 * bx + 1 < nb ? ku : 0);  // (past the last: not stored)
    const Units w[CB] = {Units(p.gate, u0), Units(p.up, u0), Units(p.gate, u1), Units(p.up, u1)};
    w4 b[D][CB];
    uint2 s[D][CB];
    uint32_t z[D][CB];
    auto load = [&](int st, int u) {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) w[cb].load(u, lane, b[st][cb], s[st][cb], z[st][cb]);
    };
#pragma unroll
    for (int st = 0; st < D; ++st)
        if (wave + WAVES * st < ku) load(st, wave + WAVES * st);
    for (int i = tid; i < ku * 16; i += WAVES * 64) {  // the row into LDS, eight k at a time: [unit][P][128]
        w4 v[P];
#pragma unroll
        for (int q = 0; q < P; ++q) v[q] = w4{};
        if (i * 8 < p.d) {
            if constexpr (F32) {
                const w4 *x = reinterpret_cast<const w4 *>(static_cast<const float *>(p.n) + (int64_t)t * p.d + i * 8);
                q4_split<P>(x[0], x[1], v);
            } else {
                v[0] = *reinterpret_cast<const w4 *>(static_cast<const uint16_t *>(p.n) + (int64_t)t * p.d + i * 8);
            }
        }
#pragma unroll
        for (int q = 0; q < P; ++q) *reinterpret_cast<w4 *>(xs + ((i >> 4) * P + q) * 128 + (i & 15) * 8) = v[q];
        if constexpr (!F32) {
            const float sum = unit_sum<XT == kXBF16>(v[0]);
            if ((i & 15) == 0) sums[i >> 4] = sum;
        }
    }
    __syncthreads();
    const int mine = (lane & 15) < P ? lane & 15 : P - 1;  // the part that the lane brings
    float acc[CB] = {};
    for (int u = wave; u < ku; u += WAVES * D) {
#pragma unroll
        for (int st = 0; st < D; ++st) {
            const int at = u + WAVES * st;
            if (at < ku) {
                few_unit<XT, CB>(xs + (at * P + mine) * 128 + 8 * h, sums + at, 0, b[st], s[st], z[st], 1.0f, acc);
                if (at + WAVES * D < ku) load(st, at + WAVES * D);
            }
        }
    }
    if (h == 0) {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) red[wave][cb * 16 + lane] = acc[cb];
    }
    __syncthreads();
    if (tid >= 32 || col >= p.f) return;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int q = 0; q < WAVES; ++q) g += red[q][(tid >> 4) * 32 + (tid & 15)], u += red[q][(tid >> 4) * 32 + 16 + (tid & 15)];
    if (!__builtin_isfinite(g) || !__builtin_isfinite(u)) {
        g = q4_slow_row<XT>(p.n, t, few_view(p.gate, p.E, p.f, p.d), e, col);
        u = q4_slow_row<XT>(p.n, t, few_view(p.up, p.E, p.f, p.d), e, col);
    }
    uint16_t part[PH];
    q4_parts<PH>(g / (1.0f + expf(-g)) * u, part);
#pragma unroll
    for (int q = 0; q < PH; ++q)
        __hip_atomic_store(out + q * kh * 128, part[q] == kNoH ? (uint16_t)0x7fc0u : part[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// y of 16 columns of a token; false (for all threads): some of h was not there.
template <int XT, int DT, bool RES>
__device__ __forceinline__ bool down_task(const FewCall &p, int t, int bx, const int32_t *chosen, const float *weights, uint16_t *xs,
                                          float *sums, float (*red)[16]) {
    constexpr int P = XT == kXF32x3 ? 3 : 2, D = 8, WAVES = kFewWaves;  // D: units ahead
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ku = (p.f + 127) >> 7, nb = (p.d + 15) >> 4, k = p.k, col = bx * 16 + tid;
    const int slots = lane < k ? chosen[t * k + lane] : -1;  // lane j: slot j's expert and weight
    const int parts = lane < k ? __builtin_bit_cast(int, weights[t * k + lane]) : 0;
    // the wave's items, a slot and a unit each: the unit goes on by eight, and over into the next slots
    struct Item {
        int j, u;
        __device__ void settle(int ku) {
            while (u >= ku) u -= ku, ++j;
        }
    };
    Item next{0, wave};
    next.settle(ku);
    Item now = next;
    w4 b[D];
    uint2 s[D];
    uint32_t z[D];
    auto load = [&](int st) {
        if (next.j < k) {
            const int e = __builtin_amdgcn_readlane(slots, next.j);
            if (e >= 0) Units(p.down, ((int64_t)e * nb + bx) * ku).load(next.u, lane, b[st], s[st], z[st]);
            next.u += WAVES;
            next.settle(ku);
        }
    };
#pragma unroll
    for (int st = 0; st < D; ++st) load(st);
    uint32_t residual = 0;  // its bits, on their way
    if constexpr (RES) {
        if (tid < 16 && col < p.d) residual = q4_bits<DT>(p.residual, (int64_t)t * p.d + col);
    }
    // h into LDS as it lies in memory, [slot][P][128 ku]
    const int pieces = k * P * ku * 16;
    const uint64_t *src = reinterpret_cast<const uint64_t *>(p.h + (int64_t)t * k * P * ku * 128);
    bool late = false;
    constexpr int B = 4;
    for (int i0 = tid; i0 < pieces; i0 += WAVES * 64 * B) {
        uint64_t v[B][2];
        for (int tries = 0;; ++tries) {
            bool missing = false;
#pragma unroll
            for (int q = 0; q < B; ++q) {
                const int i = i0 + q * WAVES * 64;
                if (i < pieces) {
                    v[q][0] = __hip_atomic_load(src + 2 * i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    v[q][1] = __hip_atomic_load(src + 2 * i + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                } else {
                    v[q][0] = v[q][1] = 0;
                }
            }
#pragma unroll
            for (int q = 0; q < B; ++q) missing |= has_none(v[q][0]) || has_none(v[q][1]);
            if (!missing) break;
            if (tries >= p.patience) {
                late = true;
                break;
            }
            __builtin_amdgcn_s_sleep(1);
        }
#pragma unroll
        for (int q = 0; q < B; ++q) {
            const int i = i0 + q * WAVES * 64;
            const w4 piece = {(uint32_t)v[q][0], (uint32_t)(v[q][0] >> 32), (uint32_t)v[q][1], (uint32_t)(v[q][1] >> 32)};
            if (i < pieces) *reinterpret_cast<w4 *>(xs + i * 8) = piece;
            if constexpr (XT != kXF32x3) {
                const float sum = unit_sum<true>(piece);
                if (i < pieces && (i & 15) == 0) sums[i >> 4] = sum;
            }
        }
    }
    if (__syncthreads_or(late)) return false;
    const int mine = (lane & 15) < P ? lane & 15 : P - 1;  // the part that the lane brings
    float acc[1] = {};
    while (now.j < k) {
#pragma unroll
        for (int st = 0; st < D; ++st) {
            if (now.j >= k) break;
            if (__builtin_amdgcn_readlane(slots, now.j) >= 0)
                few_unit<XT, 1>(xs + ((now.j * P + mine) * ku + now.u) * 128 + 8 * h, sums + now.j * P * ku + now.u, ku, &b[st], &s[st],
                                &z[st], __builtin_bit_cast(float, __builtin_amdgcn_readlane(parts, now.j)), acc);
            now.u += WAVES;
            now.settle(ku);
            load(st);
        }
    }
    if (h == 0) red[wave][lane] = acc[0];
    __syncthreads();
    if (tid >= 16 || col >= p.d) return true;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < WAVES; ++q) v += red[q][tid];
    if (!__builtin_isfinite(v)) {
        v = 0.0f;
#pragma unroll 1
        for (int j = 0; j < k; ++j) {
            const int e = chosen[t * k + j];
            if (e < 0) continue;
            const uint16_t *x = xs + j * P * ku * 128;
            const float dot = q4_slow_dot(few_view(p.down, p.E, p.d, p.f), e, col, [&](int c, float (&v8)[8]) {
                q4_x8<kXBF16>(x, c, v8);
#pragma unroll
                for (int q = 1; q < P; ++q) {
                    float part[8];
                    q4_x8<kXBF16>(x, q * ku * 128 + c, part);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v8[i] += part[i];
                }
            });
            v += weights[t * k + j] * dot;
        }
    }
    if constexpr (RES) v += q4_value<DT>(residual);
    store_from_float<DT>(p.y, (int64_t)t * p.d + col, v);
    return true;
}

template <int XT, int XH, int PH, int DT, bool RES>
__global__ __launch_bounds__(kFewWaves * 64, 4) void few_experts_kernel(FewCall p) {
    asm volatile("" ::"s"(p.gate.codes), "s"(p.down.zeros), "s"(p.weights));  // a value of each line
    extern __shared__ __attribute__((aligned(16))) uint16_t few_room[];  // a row, or a token's h; behind it sums by unit
    __shared__ float red[kFewWaves][64];
    __shared__ int32_t chosen[kFewSlots];
    __shared__ float weights[kFewSlots];
    const int tid = threadIdx.x, lane = tid & 63, k = p.k;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ups = p.T * k * p.gx, tasks = ups + p.T * p.dx;
    RouteArgs route{};
    route.bias = p.bias, route.E = p.E, route.k = k, route.groups = p.groups, route.keep = p.keep, route.n = p.per_group;
    route.group_top = p.flags & kFewTopTwo ? 2 : 1, route.sigmoid = p.flags & kFewSigmoid, route.renorm = p.flags & kFewRenorm;
    // every wave chooses for every eighth token; weights only where the workgroup has a down task
    float *sums = reinterpret_cast<float *>(few_room + p.room);
    const bool weigh = tasks <= (int)gridDim.x ? (int)blockIdx.x >= ups : true;
    for (int t = wave; t < p.T; t += kFewWaves) {
        const float *logits = p.logits + (int64_t)t * p.E;
        const Slot s = p.flags & kFewOne ? route_token<1>(route, logits, p.log_lanes, lane, weigh)
                                         : route_token<kFewOwn>(route, logits, p.log_lanes, lane, weigh);
        if (lane < k) {
            const int at = t * k + lane;
            chosen[at] = s.expert, weights[at] = s.weight;
            if (blockIdx.x == gridDim.x - 1) p.idx[at] = s.expert, p.weights[at] = s.weight;  // (has the last task)
        }
    }
    __syncthreads();
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
        const bool is_up = task < ups;
        const int at = task - ups, t = __builtin_amdgcn_readfirstlane(is_up ? task / (k * p.gx) : at / p.dx);
        for (bool form = is_up;; form = true) {
            if (form) {
                const int first = is_up ? task : t * k * p.gx, last = is_up ? task + 1 : (t + 1) * k * p.gx;
                for (int i = first; i < last; ++i) {
                    const int slot = __builtin_amdgcn_readfirstlane(i / p.gx);
                    up_task<XT, PH>(p, slot, t, i - slot * p.gx, __builtin_amdgcn_readfirstlane(chosen[slot]), few_room, sums, red);
                    __syncthreads();  // the rooms are free again
                }
                if (is_up) break;
            }
            const bool done = down_task<XH, DT, RES>(p, t, at - t * p.dx, chosen, weights, few_room, sums,
                                                         reinterpret_cast<float(*)[16]>(&red[0][0]));
            __syncthreads();
            if (done) break;
        }
    }
}

template <int XT, int XH, int PH, int DT>
hipError_t run(const FewCall &c, size_t lds, hipStream_t s) {
    // two workgroups to each of the 256 compute units, if there is work for them
    const int tasks = c.T * (c.k * c.gx + c.dx);
    const dim3 grid((unsigned)(tasks < 512 ? tasks : 512)), block(kFewWaves * 64);
    if (c.residual) few_experts_kernel<XT, XH, PH, DT, true><<<grid, block, lds, s>>>(c);
    else few_experts_kernel<XT, XH, PH, DT, false><<<grid, block, lds, s>>>(c);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few_experts(const FewArgs &f, const LayerArgs &a, hipStream_t s) {
    const RouteArgs &r = a.route;
    auto weight = [](const Q4View &v) { return FewWeight{v.codes, v.scales, v.zeros}; };
    FewCall c{};
    c.gate = weight(a.gate), c.up = weight(a.up), c.down = weight(a.down);
    c.n = f.n, c.residual = a.residual, c.h = static_cast<uint16_t *>(f.h), c.y = a.y, c.logits = f.logits, c.bias = r.bias;
    c.idx = r.idx, c.weights = r.weights, c.E = r.E, c.d = a.gate.K, c.f = a.gate.N, c.T = (int)a.T, c.k = r.k;
    c.gx = (a.gate.nb + 1) / 2, c.dx = a.down.nb, c.patience = f.patience;
    c.groups = r.groups, c.keep = r.keep, c.per_group = r.E / r.groups, c.log_lanes = route_log_lanes(r.groups);
    c.flags = (r.sigmoid ? kFewSigmoid : 0) | (r.renorm ? kFewRenorm : 0) | (r.group_top == 2 ? kFewTopTwo : 0) |
              (route_own(r.E, r.groups) <= 1 ? kFewOne : 0);
    const int parts = a.dtype == kF32 ? 3 : 2;
    const size_t up = q4_row_lds(a.gate.ku, a.dtype == kF32 ? 3 : 1), down = q4_row_lds((int64_t)r.k * a.down.ku, parts);
    const size_t rows = up > down ? up : down;
    const size_t lds = rows + rows / 64;  // a sum of 4 bytes to a unit of 256
    c.room = (int)(rows / 2);
    if (a.dtype == kF16) return run<kXF16, kXF32x2, 2, kF16>(c, lds, s);
    if (a.dtype == kBF16) return run<kXBF16, kXF32x2, 2, kBF16>(c, lds, s);
    return run<kXF32x3, kXF32x3, 3, kF32>(c, lds, s);
}

}  // namespace tq2
