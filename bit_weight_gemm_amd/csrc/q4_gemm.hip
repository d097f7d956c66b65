// 4-bit weights: packing, decode to f32, and the dense product's launches.
#include "q4_skinny.h"
#include "q4_tiled.h"

namespace tq2 {

namespace {

// One workgroup per block of 16 rows of an expert, its four waves taking the units in
// turn.  Lane (r, h) reads 16 bytes of row r (k = 128u + 32h .. +31), orders the nibbles
// and hands word c to lane (r, c) as its word h; the first 16 lanes also bring their
// row's scales and zeros.
// Done once per weight, before its use: 4096 x 4096 11 us, 64 x 2048 x 1024 30 us, 4.6 TB/s
// read and written, as a copy.
__global__ __launch_bounds__(256) void q4_pack_kernel(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros,
                                                      Q4View v, w4 *oc, uint16_t *os, uint8_t *oz) {
    __shared__ uint32_t words[4][16][4][4 + 1];  // [wave][r][h of the reader][word]
    const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4, wave = threadIdx.x >> 6;
    const int nb = blockIdx.x, e = blockIdx.y;
    const int n = nb * 16 + r;
    const int64_t row = (int64_t)e * v.N + n, unit0 = ((int64_t)e * v.nb + nb) * v.ku;
    const int gpu = 128 / v.G, kg = v.K / v.G;
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
                    os[((unit0 + u) * 16 + r) * gpu + g] = has ? scales[row * kg + at] : 0;
                    if (oz) oz[((unit0 + u) * 16 + r) * gpu + g] = has ? zeros[row * kg + at] : 8;
                }
        }
        __syncthreads();
    }
}

__global__ __launch_bounds__(256) void q4_dequant_kernel(Q4View v, float *out) {
    const int64_t n = (int64_t)v.E * v.N * v.K, step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
        const int k = (int)(i % v.K);
        const int64_t en = i / v.K;
        out[i] = q4_weight_at(v, (int)(en / v.N), (int)(en % v.N), k);
    }
}

}  // namespace

hipError_t launch_q4_pack(const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, const Q4View &v,
                          hipStream_t s) {
    q4_pack_kernel<<<dim3((unsigned)v.nb, (unsigned)v.E), dim3(256), 0, s>>>(
        codes, scales, zeros, v, const_cast<w4 *>(v.codes), const_cast<uint16_t *>(v.scales),
        const_cast<uint8_t *>(v.zeros));
    return hipGetLastError();
}

hipError_t launch_q4_dequant(const Q4View &v, float *out, hipStream_t s) {
    const int64_t n = (int64_t)v.E * v.N * v.K;
    const int64_t blocks = (n + 255) / 256, most = (int64_t)1 << 20;
    q4_dequant_kernel<<<dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, s>>>(v, out);
    return hipGetLastError();
}

namespace {

// How M rows are multiplied: tiles of bm rows with the units in `split` shares, or, bm 0, the
// skinny kernel on blocks of 32 rows.
struct Deal {
    int bm, split;
};

// The shortest by an estimate in microseconds, whose constants were fitted to measured times
// (M = 33 .. 2048; N x K = 4096 x 4096, 14336 x 4096, 5003 x 4000, 1024 x 1024 and 1000 x 8192;
// all G and types).  A kernel takes as many rounds of the 256 compute units as its workgroups need,
// and in each so many microseconds a unit of 128 k (without LDS a last round counts half by its
// workgroups); shares are written and joined at 8 TB/s, with more time for the launch and for rows
// that are not aligned.
// f16, 4096 x 4096, estimate against measured: 64 rows skinny 10.8 / 11.2, 128 rows in
// 8 shares 17.6 / 16.7 (skinny 19.5), 256 rows in 4 shares 23 / 21.5 (skinny 35, one share 39), 512 rows in
// 2 shares 34 / 32 (one 40), 2048 rows in tiles of 128 67 / 72 (of 64: 84).
Deal deal(int64_t N, int64_t K, int64_t G, int64_t M, int dtype) {
    if (M <= 32) return Deal{0, 1};  // 4096 x 4096: 10 us, in tiles at least 14
    constexpr double kCus = 256;
    const bool f32 = dtype == kF32, fine = G == 32;
    const double nb = (double)((N + 15) / 16), ku = (double)((K + 127) / 128);
    auto up = [](double v) { return (double)(int64_t)(v + 0.999999); };
    Deal best{0, 1};
    double least = 1e300;
    if (M <= 65535 * 32) {  // a grid's second axis
        const double blocks = up(nb / 2), rows = (double)((M + 31) / 32);
        double wk = 1;
        while (wk < 8 && blocks * rows * wk < kWavesWanted && 2 * wk <= ku) wk *= 2;
        const double full = up(blocks * wk / 8) * rows / kCus, share = full <= 1 ? 1 : (full + up(full)) / 2;
        least = share * (2.0 + up(ku / wk) * (f32 ? (fine ? 4.5 : 3.9) : (fine ? 2.6 : 2.2)));
    }
    for (int bm = 64; bm <= 128; bm *= 2) {
        if (bm == 128 && f32 && fine) continue;  // its registers do not suffice
        const double tiles = up(nb / 16) * up((double)M / bm);
        const double unit = f32 ? (bm == 64 ? (fine ? 2.4 : 2.0) : 3.4) : (bm == 64 ? (fine ? 1.6 : 1.35) : (fine ? 2.4 : 1.95));
        for (int split = 1; split <= 16 && split <= ku && (split == 1 || tiles * split <= kCus); ++split) {
            const double us = 5.5 + (q4_plain_x(K, dtype) ? 0.0 : 5.0) + up(tiles * split / kCus) * up(ku / split) * unit +
                              (split == 1 ? 0.0 : (N % 4 ? 6.5 : 3.5) + (double)split * M * N * 1e-6);
            if (us < least) least = us, best = Deal{bm, split};
        }
    }
    return best;
}

struct DenseWs {
    size_t off_scale, off_part, total;
    int64_t part_stride;
};
DenseWs dense_ws(const Deal &d, int64_t N, int64_t K, int64_t M, int dtype) {
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    DenseWs w{};
    const bool plain = q4_plain_x(K, dtype);
    w.off_scale = plain ? 0 : up((size_t)q4_planes(dtype) * M * ((K + 127) / 128 * 128) * 2);
    w.off_part = w.off_scale + (plain ? 0 : up((size_t)M * 4));
    w.part_stride = (M * N + 3) / 4 * 4;
    w.total = w.off_part + (d.split > 1 ? (size_t)d.split * w.part_stride * 4 : 0);
    return w;
}

}  // namespace

size_t q4_gemm_workspace(int64_t N, int64_t K, int64_t G, int64_t M, int dtype) {
    const Deal d = deal(N, K, G, M, dtype);
    return d.bm ? dense_ws(d, N, K, M, dtype).total : 0;
}

hipError_t launch_q4_gemm(const Q4View &v, const void *x, void *y, int64_t M, int dtype, void *ws, const Q4Epilogue *epi,
                          hipStream_t s) {
    const Deal d = deal(v.N, v.K, v.G, M, dtype);
    if (d.bm) {
        const DenseWs w = dense_ws(d, v.N, v.K, M, dtype);
        char *b = static_cast<char *>(ws);
        Q4TArgs a{};
        a.w = v, a.y = y, a.M = M, a.split = d.split;
        if (q4_plain_x(v.K, dtype)) {
            a.a = static_cast<const _Float16 *>(x), a.lda = v.K;
        } else {
            Q4Prep p{};
            p.x = x, p.rows = M, p.K = v.K;
            p.lda = (int64_t)v.ku * 128, p.plane = M * p.lda;
            p.out = reinterpret_cast<_Float16 *>(b);
            p.rowscale = reinterpret_cast<float *>(b + w.off_scale);
            const hipError_t e = launch_q4_prep(p, dtype, s);
            if (e != hipSuccess) return e;
            a.a = p.out, a.lda = p.lda, a.plane = p.plane, a.rowscale = p.rowscale;
        }
        if (d.split > 1) a.part = reinterpret_cast<float *>(b + w.off_part), a.part_stride = w.part_stride;
        if (epi) a.epi = *epi;
        // shares are joined first: their products are q4_gemm's own
        const hipError_t e = epi && d.split == 1 ? launch_q4_tiled_epilogue(a, dtype, d.bm, s) : launch_q4_tiled_dense(a, dtype, d.bm, s);
        if (e != hipSuccess || d.split == 1) return e;
        if (epi) return launch_q4_join_epilogue(a, y, dtype, s);
        return launch_q4_join(a.part, a.part_stride, d.split, y, M * v.N, dtype, s);
    }
    Q4Args a{};
    a.w = v, a.x = x, a.y = y, a.M = M;
    if (!epi) return q4_dense<false>(a, dtype, s);
    a.epi = *epi;
    return launch_q4_dense_epilogue(a, dtype, s);
}

}  // namespace tq2
