// 4-bit weights: packing, decode to f32, and the dense product's launches.
#include "q4_skinny.h"
#include "q4_tiled.h"

namespace tq2 {

namespace {

__global__ __launch_bounds__(1024) void q4_head_kernel(uint32_t *head, int E) {
    if ((int)threadIdx.x < E) head[threadIdx.x] = 0;
}

// One thread per lane of a unit: its four words, each from four consecutive bytes of
// the row-major codes; the first 16 lanes also bring their row's scales and zeros.
// The head collects each expert's largest |scale| (integer maximum: the order does not matter).
__global__ __launch_bounds__(256) void q4_pack_kernel(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros,
                                                      Q4View v, w4 *oc, uint16_t *os, uint8_t *oz, uint32_t *head,
                                                      int64_t units) {
    const int64_t gid = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t unit = gid >> 6;
    const int lane = gid & 63, r = lane & 15, h = lane >> 4;
    uint32_t most = 0;
    if (unit < units) {
        const int u = (int)(unit % v.ku);
        const int64_t eb = unit / v.ku;
        const int nb = (int)(eb % v.nb);
        const int64_t e = eb / v.nb;
        const int n = nb * 16 + r;
        w4 out = {0, 0, 0, 0};
        const int64_t row = e * v.N + n;
        if (n < v.N) {
            for (int j = 0; j < 4; ++j) {
                const int k = u * 128 + 32 * j + 8 * h;
                if (k >= v.K) break;
                const uint32_t b = *reinterpret_cast<const uint32_t *>(codes + (row * v.K + k) / 2);
                uint32_t w = 0;
                for (int s = 0; s < 4; ++s)
                    w |= ((b >> (8 * s)) & 15u) << (4 * s) | ((b >> (8 * s + 4)) & 15u) << (16 + 4 * s);
                out[j] = w;
            }
        }
        oc[gid] = out;
        if (h == 0) {
            const int gpu = 128 / v.G, kg = v.K / v.G;
            for (int g = 0; g < gpu; ++g) {
                const int kgi = u * gpu + g;
                const bool in = n < v.N && kgi < kg;
                const uint16_t s = in ? scales[row * kg + kgi] : 0;
                os[(unit * 16 + r) * gpu + g] = s;
                if (oz) oz[(unit * 16 + r) * gpu + g] = in ? zeros[row * kg + kgi] : 8;
                const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_fabsf(half_bits(s)));
                most = a > most ? a : most;
            }
        }
    }
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t b = (uint32_t)__shfl_xor((int)most, o);
        most = b > most ? b : most;
    }
    if (lane == 0 && most) atomicMax(&head[unit / v.ku / v.nb], most);
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
    // Column blocks per workgroup: one while that fits the 256 compute units in one
    // round of workgroups, more beyond, so that x is read less often.
    const int64_t nb = a.w.nb;
    if (a.M <= 16) {
        if (nb <= 512) return run_q4_skinny<XT, G, 1, 1, kDense>(a, 1, s);
        if (nb <= 1024) return run_q4_skinny<XT, G, 1, 2, kDense>(a, 1, s);
        return run_q4_skinny<XT, G, 1, 4, kDense>(a, 1, s);
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
    const int64_t units = (int64_t)v.E * v.nb * v.ku;
    q4_pack_kernel<<<dim3((unsigned)((units + 3) / 4)), dim3(256), 0, s>>>(
        codes, scales, zeros, v, const_cast<w4 *>(v.codes), const_cast<uint16_t *>(v.scales),
        const_cast<uint8_t *>(v.zeros), head, units);
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
