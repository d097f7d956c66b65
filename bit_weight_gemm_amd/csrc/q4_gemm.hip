// 4-bit weights: packing, decode to f32, and the dense product's launches.
#include "q4_skinny.h"
#include "q4_tiled.h"

namespace tq2 {

namespace {

__global__ __launch_bounds__(1024) void q4_head_kernel(uint32_t *head, int E) {
    if ((int)threadIdx.x < E) head[threadIdx.x] = 0;
}

// One workgroup per block of 16 rows of an expert, its four waves taking the units in
// turn.  Lane (r, h) reads 16 bytes of row r (k = 128u + 32h .. +31), orders the nibbles
// and hands word c to lane (r, c) as its word h; the first 16 lanes also bring their
// row's scales and zeros.  The head collects each expert's largest |scale| (integer
// maximum: the order does not matter), which a wave adds to only where it is larger.
__global__ __launch_bounds__(256) void q4_pack_kernel(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros,
                                                      Q4View v, w4 *oc, uint16_t *os, uint8_t *oz, uint32_t *head) {
    __shared__ uint32_t words[4][16][4][4 + 1];  // [wave][r][h of the reader][word]
    const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4, wave = threadIdx.x >> 6;
    const int nb = blockIdx.x, e = blockIdx.y;
    const int n = nb * 16 + r;
    const int64_t row = (int64_t)e * v.N + n, unit0 = ((int64_t)e * v.nb + nb) * v.ku;
    const int gpu = 128 / v.G, kg = v.K / v.G;
    uint32_t most = 0;
    for (int u0 = 0; u0 < v.ku; u0 += 4) {
        const int u = u0 + wave;
        const int k = u * 128 + 32 * h;  // K is a multiple of 32: whole pieces
        w4 in = {0, 0, 0, 0};
        if (n < v.N && u < v.ku && k < v.K) {
            const uint32_t *b = reinterpret_cast<const uint32_t *>(codes + (row * v.K + k) / 2);
            in = w4{b[0], b[1], b[2], b[3]};
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t w = 0;
#pragma unroll
            for (int s = 0; s < 4; ++s)
                w |= ((in[c] >> (8 * s)) & 15u) << (4 * s) | ((in[c] >> (8 * s + 4)) & 15u) << (16 + 4 * s);
            words[wave][r][h][c] = w;
        }
        __syncthreads();
        if (u < v.ku) {
            oc[(unit0 + u) * 64 + lane] = w4{words[wave][r][0][h], words[wave][r][1][h], words[wave][r][2][h], words[wave][r][3][h]};
            if (h == 0)
                for (int g = 0; g < gpu; ++g) {
                    const int at = u * gpu + g;
                    const bool has = n < v.N && at < kg;
                    const uint16_t s = has ? scales[row * kg + at] : 0;
                    os[((unit0 + u) * 16 + r) * gpu + g] = s;
                    if (oz) oz[((unit0 + u) * 16 + r) * gpu + g] = has ? zeros[row * kg + at] : 8;
                    const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_fabsf(half_bits(s)));
                    most = a > most ? a : most;
                }
        }
        __syncthreads();
    }
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t b = (uint32_t)__shfl_xor((int)most, o);
        most = b > most ? b : most;
    }
    if (lane == 0 && most > *const_cast<volatile uint32_t *>(&head[e])) atomicMax(&head[e], most);
}

__global__ __launch_bounds__(256) void q4_dequant_kernel(Q4View v, float *out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)v.E * v.N * v.K) return;
    const int k = (int)(i % v.K);
    const int64_t en = i / v.K;
    out[i] = q4_weight_at(v, (int)(en / v.N), (int)(en % v.N), k);
}

template <int XT, int G>
hipError_t dense(const Q4Args &a, hipStream_t s) {
    // Column blocks per wave: one while that fits the 256 compute units in two
    // rounds of workgroups, more beyond, so that x is read less often.
    const int64_t nb = a.w.nb;
    if (a.M <= 16) {
        if (nb <= 512) return run_q4_skinny<XT, G, 1, 1, kDense>(a, 1, s);
        return run_q4_skinny<XT, G, 1, 2, kDense>(a, 1, s);
    }
    if (a.M <= 32 || XT == kXF32x3) return run_q4_skinny<XT, G, 2, 2, kDense>(a, (a.M + 31) / 32, s);
    return run_q4_skinny<XT, G, 4, 2, kDense>(a, (a.M + 63) / 64, s);
}

template <int XT>
hipError_t dense_g(const Q4Args &a, hipStream_t s) {
    if (a.w.G == 32) return dense<XT, 32>(a, s);
    if (a.w.G == 64) return dense<XT, 64>(a, s);
    return dense<XT, 128>(a, s);
}

}  // namespace

hipError_t launch_q4_pack(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, const Q4View &v,
                          hipStream_t s) {
    uint32_t *head = const_cast<uint32_t *>(v.head);
    q4_head_kernel<<<dim3(1), dim3(1024), 0, s>>>(head, v.E);
    q4_pack_kernel<<<dim3((unsigned)v.nb, (unsigned)v.E), dim3(256), 0, s>>>(
        codes, scales, zeros, v, const_cast<w4 *>(v.codes), const_cast<uint16_t *>(v.scales),
        const_cast<uint8_t *>(v.zeros), head);
    return hipGetLastError();
}

hipError_t launch_q4_dequant(const Q4View &v, float *out, hipStream_t s) {
    const int64_t n = (int64_t)v.E * v.N * v.K;
    q4_dequant_kernel<<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s>>>(v, out);
    return hipGetLastError();
}

// The tiled product from kTiledRows rows on (below, the skinny kernel on tiles of 64).
constexpr int64_t kTiledRows = 256;

size_t q4_gemm_workspace(int64_t, int64_t K, int64_t M, int dtype) {
    if (M < kTiledRows || q4_plain_x(K, dtype)) return 0;
    const size_t lda = (size_t)(K + 127) / 128 * 128;
    return (size_t)q4_planes(dtype) * M * lda * 2 + (size_t)(M * 4 + 255) / 256 * 256;
}

hipError_t launch_q4_gemm(const Q4View &v, const void *x, void *y, int64_t M, int dtype, void *ws, hipStream_t s) {
    if (M >= kTiledRows) {
        Q4TArgs a{};
        a.w = v, a.y = y, a.M = M;
        if (q4_plain_x(v.K, dtype)) {
            a.a = static_cast<const _Float16 *>(x), a.lda = v.K;
        } else {
            Q4Prep p{};
            p.x = x, p.rows = M, p.K = v.K;
            p.lda = (int64_t)v.ku * 128, p.plane = M * p.lda;
            p.out = static_cast<_Float16 *>(ws);
            p.rowscale = reinterpret_cast<float *>(p.out + q4_planes(dtype) * p.plane);
            const hipError_t e = launch_q4_prep(p, dtype, s);
            if (e != hipSuccess) return e;
            a.a = p.out, a.lda = p.lda, a.plane = p.plane, a.rowscale = p.rowscale;
        }
        return launch_q4_tiled_dense(a, dtype, 128, s);
    }
    Q4Args a{};
    a.w = v, a.x = x, a.y = y, a.M = M;
    if (dtype == kF16) return dense_g<kXF16>(a, s);
    if (dtype == kBF16) return dense_g<kXBF16>(a, s);
    return dense_g<kXF32x3>(a, s);
}

}  // namespace tq2
