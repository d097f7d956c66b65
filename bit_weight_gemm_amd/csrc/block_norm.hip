// The norms after and before a block, with its gate and residual scale, and their gradient:
//   u = norm(b) post + post_bias (b itself without post)
//   y = x + scale gate u, rounded to its type
//   n = norm(y) pre + pre_bias
// with norm(v) = v / sqrt(mean(v^2) + eps), or (v - mean) / sqrt(var + eps).
//
// One pass over memory: TPR threads hold a row (C pieces of 16 bytes each), every input is read once, sums go over the
// wave by lane exchanges and over the waves through LDS.
// Bound by memory where a thread has eight columns or fewer: 4096 x 4096 bf16, three sets of inputs in turn, forward 33 us (134 MB,
// 4.1 TB/s; a large copy reaches 5.1), gradient 54 us (201 MB and 25 MB of parts, 4.2 TB/s), f32 53 and 89 us; one row 3.6 and 8.1 us
// (launches).  With means 50-54 and 84 us: their f64 sums and differences.  Narrower rows: 4096 x 1024 bf16 11.5 and 28 us (a row's
// threads are a whole workgroup in the gradient).  Longer ones (more than 4096 columns) have more of a row to a thread than its
// registers hold.  Forward: 2048 x 8192 bf16 43 us (3.1 TB/s), with means 53; 60 to 988 bytes a lane of scratch beyond 8192 columns (f32 with
// means beyond 4096): 1000 x 16384 bf16 44.  Gradient, scratch of 440 bytes a lane and more, up to 3240: 2048 x 5000 bf16 146 us (0.8 TB/s),
// 2048 x 8192 161 (1.3 TB/s), with means 295, 1000 x 16384 443; f32, 2048 x 5120, 301, 1000 x 8192 185.
#include "block_norm.h"

namespace tq2 {

namespace {

// Threads of a workgroup: rows of one wave share workgroups of four.
constexpr int threads_of(int tpr) { return tpr == 64 ? 256 : tpr; }

// FULL: with means or biases.  The rows go round the workgroups.  Parameters that are the same for all rows stay in registers, and the next row's pieces are on
// their way while one is normed.
template <int DT, int WT, int TPR, int C, int MODE, bool FULL>
__global__ __launch_bounds__(threads_of(TPR)) void block_norm_kernel(BlockNormArgs p) {
    constexpr int V = kPiece<DT>, ROWS = threads_of(TPR) / TPR;
    constexpr bool HOLD = C * V <= 8;  // (more of everything would not fit)
    __shared__ double room[2][TPR / 64 * 2];
    __shared__ double far_room[FULL ? TPR / 64 : 1];  // (its uses lie between those of the other two: one is enough)
    const int tid = threadIdx.x % TPR, N = p.N;
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t row = (int64_t)blockIdx.x * ROWS + __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
    Raw<DT, V> x[C], b[C];
    Raw<WT, V> post[C], gate[C], pre[C], post_bias[C], pre_bias[C];
    auto piece = [&](int c) { return Piece<V, MODE>(tid + TPR * c, N); };
    auto rows = [&](int64_t r) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (p.b) piece(c).template load<DT>(p.b, r * N, N, b[c]);
            piece(c).template load<DT>(p.x, r * N, N, x[c]);
        }
    };
    auto vector = [&](const void *from, int64_t at, Raw<WT, V> (&to)[C]) {
        if (from)
#pragma unroll
            for (int c = 0; c < C; ++c) piece(c).template load<WT>(from, at, N, to[c]);
    };
    const bool one_gate = p.gate_rows == p.M;
    if (row < p.M) rows(row);
    if constexpr (HOLD) {
        vector(p.post, 0, post), vector(p.post_bias, 0, post_bias), vector(p.pre, 0, pre), vector(p.pre_bias, 0, pre_bias);
        if (one_gate) vector(p.gate, 0, gate);
    }
    // sums of a row's values (for FULL) and of their squares, and the norm of that
    auto norm = [&](const float (&v)[C][V], double *where) {
        double sum[2] = {};
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const double w = v[c][q];
                sum[0] = __builtin_fma(w, w, sum[0]);
                if constexpr (FULL) sum[1] += w;
            }
        row_total<TPR, FULL ? 2 : 1>(reinterpret_cast<double(&)[FULL ? 2 : 1]>(sum), where);
        Norm r = norm_of(sum[1], sum[0], N, p.layer, p.eps);
        if constexpr (FULL) {
            if (p.layer && is_far(r)) {  // (the same for all threads of the row) the squares again, of the differences
                double again[1] = {};
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int q = 0; q < V; ++q) {
                        const double w = q < piece(c).left ? (double)v[c][q] - r.mean : 0.0;
                        again[0] = __builtin_fma(w, w, again[0]);
                    }
                row_total<TPR, 1>(again, far_room);
                r.rstd = norm_of(0.0, again[0], N, true, p.eps).rstd;
            }
        }
        return r;
    };
    auto scaled = [&](const Norm &r, float (&v)[C][V], const Raw<WT, V> (&weight)[C], bool biased, const Raw<WT, V> (&bias)[C]) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float w[V], k[V] = {};
            piece(c).template values<WT>(weight[c], w);
            if (FULL && biased) piece(c).template values<WT>(bias[c], k);
#pragma unroll
            for (int q = 0; q < V; ++q) v[c][q] = norm_value<FULL>(r, v[c][q], w[q], k[q]);
        }
    };
    for (; row < p.M; row += step) {
        const int64_t at = row * N;
        float y[C][V], u[C][V];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            piece(c).template values<DT>(x[c], y[c]);
            if (p.b) piece(c).template values<DT>(b[c], u[c]);
        }
        if (!one_gate) vector(p.gate, row / p.gate_rows * N, gate);
        if (row + step < p.M) rows(row + step);
        if (p.b) {
            if (p.post) {
                if constexpr (!HOLD) vector(p.post, 0, post), vector(p.post_bias, 0, post_bias);
                scaled(norm(u, room[0]), u, post, p.post_bias != nullptr, post_bias);
            }
            if constexpr (!HOLD) {
                if (one_gate) vector(p.gate, 0, gate);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float g[V];
                if (p.gate) piece(c).template values<WT>(gate[c], g);
#pragma unroll
                for (int q = 0; q < V; ++q)
                    y[c][q] = rounded<DT>(y[c][q] + p.scale * (p.gate ? g[q] : 1.0f) * u[c][q]);
                if (p.y) piece(c).template store<DT>(p.y, at, y[c]);
            }
        }
        if (p.n) {
            if constexpr (!HOLD) vector(p.pre, 0, pre), vector(p.pre_bias, 0, pre_bias);
            scaled(norm(y, room[1]), y, pre, p.pre_bias != nullptr, pre_bias);
#pragma unroll
            for (int c = 0; c < C; ++c) piece(c).template store<DT>(p.n, at, y[c]);
        }
        if (TPR > 64 && !(p.b && p.post && p.n)) __syncthreads();  // one of the rooms is used twice in a row
    }
}

// ---- gradient
//
// dn and dy are the gradients of n and y.  With y^ = norm(y), g = dn pre and std its divisor,
//   dY = dy + (g - y^ mean(g y^) [- mean(g)]) / std,  dx = dY,
//   dpre = sum over rows of dn y^, dpre_bias of dn,
//   dgate = scale sum over its rows of u dY,  du = scale gate dY (db, without post),
//   dpost = sum of du b^, dpost_bias of du,  db as above from du post and b^.
// mean(g y^) is formed from sums of g y, so that a row needs two rounds of sums: its squares' and those, then du's.
// The sums over rows are kept in f32 by the workgroup that has the rows, in registers, and written as one part each;
// a second kernel adds the parts in their order.

// Workgroups: `parts` to each run of rows that share a gate, or whole runs to a workgroup.
struct Shares {
    int64_t groups, parts;   // runs of rows with one gate; workgroups of a run (1: whole runs, dealt round)
    int64_t workers;         // workgroups
};
// Threads of a row: of its pieces, a power of two from one wave to 512.  (1024 threads have 128 registers each: 2048 rows of 8192, bf16,
// took 228 us instead of 154, 4096 rows of 4096, f32, 254 instead of 89.)
constexpr int kMostThreads = 512;
int row_threads(int64_t N, int dtype) {
    const int64_t pieces = (N + (dtype == kF32 ? 3 : 7)) / (dtype == kF32 ? 4 : 8);
    int t = 64;
    while (t < pieces && t < kMostThreads) t *= 2;
    return t;
}
Shares shares_of(int64_t M, int64_t N, int64_t R, int dtype) {
    const int threads = row_threads(N, dtype);
    const int64_t want = threads == 64 ? 1024 : threads < 512 ? 512 : 256;
    Shares s;
    s.groups = R;
    const int64_t run = M / R;
    s.parts = R >= want ? 1 : want / R;
    if (s.parts > run) s.parts = run;
    s.workers = s.parts > 1 || R <= want ? R * s.parts : want;
    return s;
}

// V floats from column `col` of N on.
template <int V>
__device__ __forceinline__ void put_floats(float *row, int col, int N, const float (&v)[V]) {
    if (col + V <= N) {
        __builtin_memcpy(row + col, v, V * 4);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (col + i < N) row[col + i] = v[i];
    }
}

template <int DT, int WT, int TPR, int C, int MODE, bool FULL>
__global__ __launch_bounds__(TPR) void block_norm_backward_kernel(BlockNormBackwardArgs p, Shares s) {
    constexpr int V = kPiece<DT>, S0 = FULL ? 2 : 0, S1 = FULL ? 6 : 3, S2 = FULL ? 2 : 1;
    constexpr bool HOLD = C * V <= 8;  // parameters stay in registers, and the next row's pieces are on their way
    __shared__ double room[2][TPR / 64 * (S0 + S1 + S2)];  // by turns: a row's sums are read while the next one's are written
    const int tid = threadIdx.x, N = p.N;
    auto piece = [&](int c) { return Piece<V, MODE>(tid + TPR * c, N); };
    float dpre[C][V] = {}, dpost[C][V] = {};
    float dpre_bias[FULL ? C : 1][FULL ? V : 1] = {}, dpost_bias[FULL ? C : 1][FULL ? V : 1] = {};
    Raw<DT, V> ry[C], rb[C], rdy[C], rdn[C];
    Raw<WT, V> pre[C], post[C], post_bias[C], gate[C];
    auto rows = [&](int64_t row) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t at = row * N;
            if (p.pre) piece(c).template load<DT>(p.y, at, N, ry[c]), piece(c).template load<DT>(p.dn, at, N, rdn[c]);
            if (p.b) piece(c).template load<DT>(p.b, at, N, rb[c]);
            if (p.dy) piece(c).template load<DT>(p.dy, at, N, rdy[c]);
        }
    };
    auto vector = [&](const void *from, int64_t at, Raw<WT, V> (&to)[C]) {
        if (from)
#pragma unroll
            for (int c = 0; c < C; ++c) piece(c).template load<WT>(from, at, N, to[c]);
    };
    const int64_t run = p.gate_rows;
    int turn = 0;
    if constexpr (HOLD) vector(p.pre, 0, pre), vector(p.post, 0, post), vector(p.post_bias, 0, post_bias);
    for (int64_t job = blockIdx.x; job < s.groups * s.parts; job += gridDim.x) {
        const int64_t group = job / s.parts, part = job % s.parts;
        const int64_t r0 = group * run + run * part / s.parts, r1 = group * run + run * (part + 1) / s.parts;
        float dgate[C][V] = {};
        if constexpr (HOLD) vector(p.gate, group * N, gate);
        if (HOLD && r0 < r1) rows(r0);
        for (int64_t row = r0; row < r1; ++row, turn ^= 1) {
            const int64_t at = row * N;
            float y[C][V], b[C][V], d[C][V], dn[C][V], w[V], mb = 0.0f;
            if constexpr (!HOLD) rows(row);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (p.pre) piece(c).template values<DT>(ry[c], y[c]), piece(c).template values<DT>(rdn[c], dn[c]);
                if (p.b) piece(c).template values<DT>(rb[c], b[c]);
                if (p.dy) piece(c).template values<DT>(rdy[c], d[c]);
                else
#pragma unroll
                    for (int i = 0; i < V; ++i) d[c][i] = 0.0f;
            }
            if constexpr (HOLD) {
                if (row + 1 < r1) rows(row + 1);
            } else {
                vector(p.pre, 0, pre);
            }
            // Where means count, y and b are first brought near theirs, by sums that need not be exact: what is left of the means
            // comes out of the sums behind.
            if constexpr (FULL) {
                double sum[2] = {};
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (p.pre) a0 += y[c][i];
                        if (p.post) a1 += b[c][i];
                    }
                    sum[0] += a0, sum[1] += a1;
                }
                row_total<TPR, 2>(sum, room[turn]);
                if (p.layer) {
                    const float my = (float)(sum[0] / N);
                    mb = (float)(sum[1] / N);
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const bool in = MODE == kWhole ? piece(c).any() : i < piece(c).left;
                            y[c][i] = in ? y[c][i] - my : 0.0f;
                            if (p.post) b[c][i] = in ? b[c][i] - mb : 0.0f;
                        }
                }
            }
            // squares of y and b in f64, for their range, and g y; where means count, also y and b (in f64: y^ may lie at 0) and g
            double sum[S1] = {};
            if (p.pre) {
                float gy = 0.0f, g0 = 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    piece(c).template values<WT>(pre[c], w);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float g = dn[c][i] * w[i];
                        const double v = y[c][i];
                        sum[0] = __builtin_fma(v, v, sum[0]);
                        gy += g * y[c][i];
                        if constexpr (FULL) sum[3] += v, g0 += g;
                    }
                }
                sum[2] = gy;
                if constexpr (FULL) sum[5] = g0;
            }
            if (p.post) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const double v = b[c][i];
                        sum[1] = __builtin_fma(v, v, sum[1]);
                        if constexpr (FULL) sum[4] += v;
                    }
                }
            }
            row_total<TPR, S1>(sum, room[turn] + TPR / 64 * S0);
            if (p.pre) {
                const Norm r = norm_of(FULL ? sum[FULL ? 3 : 0] : 0.0, sum[0], N, p.layer, p.eps);
                const float rstd = (float)r.rstd, mean = (float)r.mean;
                // mean(g y^) and mean(g)
                const float m1 = (float)((FULL ? sum[2] - r.mean * sum[FULL ? 5 : 0] : sum[2]) * r.rstd / N);
                const float m0 = FULL && p.layer ? (float)(sum[FULL ? 5 : 0] / N) : 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    piece(c).template values<WT>(pre[c], w);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float hat = (FULL ? y[c][i] - mean : y[c][i]) * rstd;
                        dpre[c][i] += dn[c][i] * hat;
                        if constexpr (FULL) dpre_bias[c][i] += dn[c][i];
                        d[c][i] += (dn[c][i] * w[i] - m0 - hat * m1) * rstd;
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (p.dx) piece(c).template store<DT>(p.dx, at, d[c]);
            if (!p.b) {
                continue;
            }
            // (past the row's end d is whatever m0 and m1 make of zeros, and counts nowhere: b^, the weights, the gate or a store hold it back)
            if (p.post) {
                if constexpr (!HOLD) vector(p.post, 0, post), vector(p.post_bias, 0, post_bias), vector(p.gate, group * N, gate);
                const Norm r = norm_of(FULL ? sum[FULL ? 4 : 0] : 0.0, sum[1], N, p.layer, p.eps);
                const float rstd = (float)r.rstd, mean = (float)r.mean;
                double gs[S2] = {};
                float gb = 0.0f, g0 = 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float k[V] = {}, gv[V];
                    piece(c).template values<WT>(post[c], w);
                    if (FULL && p.post_bias) piece(c).template values<WT>(post_bias[c], k);
                    if (p.gate) piece(c).template values<WT>(gate[c], gv);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float hat = (FULL ? b[c][i] - mean : b[c][i]) * rstd;
                        dgate[c][i] += (FULL ? hat * w[i] + k[i] : hat * w[i]) * d[c][i];
                        const float du = p.scale * (p.gate ? gv[i] : 1.0f) * d[c][i];
                        dpost[c][i] += du * hat;
                        if constexpr (FULL) dpost_bias[c][i] += du;
                        b[c][i] = hat;
                        d[c][i] = du * w[i];  // (w is 0 past the row's end)
                        gb += d[c][i] * hat;
                        if constexpr (FULL) g0 += d[c][i];
                    }
                }
                gs[0] = gb;
                if constexpr (FULL) gs[1] = g0;
                row_total<TPR, S2>(gs, room[turn] + TPR / 64 * (S0 + S1));
                const float m1 = (float)gs[0] / N, m0 = FULL && p.layer ? (float)gs[S2 - 1] / N : 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < V; ++i) d[c][i] = (d[c][i] - m0 - b[c][i] * m1) * rstd;
            } else {
                if constexpr (!HOLD) vector(p.gate, group * N, gate);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float gv[V];
                    if (p.gate) piece(c).template values<WT>(gate[c], gv);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        dgate[c][i] += b[c][i] * d[c][i];
                        d[c][i] *= p.scale * (p.gate ? gv[i] : 1.0f);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (p.db) piece(c).template store<DT>(p.db, at, d[c]);
        }
        if (p.dgate) {  // scaled here: the parts are sums of finished terms
            float *out = s.parts == 1 ? p.dgate : p.part + (int64_t)gridDim.x * 4 * N;
#pragma unroll
            for (int c = 0; c < C; ++c) {
#pragma unroll
                for (int i = 0; i < V; ++i) dgate[c][i] *= p.scale;
                put_floats<V>(out + job * N, (tid + TPR * c) * V, N, dgate[c]);
            }
        }
    }
    auto put = [&](bool asked, int which, const auto &v) {
        if (!asked) return;
        float *out = p.part + ((int64_t)which * gridDim.x + blockIdx.x) * N;
#pragma unroll
        for (int c = 0; c < C; ++c) put_floats<V>(out, (tid + TPR * c) * V, N, v[c]);
    };
    put(p.dpre, 0, dpre), put(p.dpost, 2, dpost);
    if constexpr (FULL) put(p.dpre_bias, 1, dpre_bias), put(p.dpost_bias, 3, dpost_bias);
}

// out[which][n] = the sum of `count` parts, in an order that depends on their number alone: 64 threads take every 64th each
// of four columns, and their sums are added in pairs.
struct PartSum {
    const float *part;
    float *out;
    int64_t count;
};
struct PartSums {
    PartSum s[4];
    const float *gate_part;
    float *dgate;
    int64_t gate_parts;
    int N;
};
__global__ __launch_bounds__(1024) void block_norm_parts_kernel(PartSums p) {
    __shared__ float sums[64][64];
    const int share = threadIdx.x >> 4, own = threadIdx.x & 15;
    const Piece<4, kShort> at(blockIdx.x * 16 + own, p.N);
    PartSum s;
    if (blockIdx.y < 4) s = p.s[blockIdx.y];
    else s = PartSum{p.gate_part + (int64_t)(blockIdx.y - 4) * p.gate_parts * p.N, p.dgate + (int64_t)(blockIdx.y - 4) * p.N,
                     p.gate_parts};
    if (!s.out) return;  // the whole workgroup
    float v[4] = {};
    if (at.full()) {
#pragma unroll 4
        for (int64_t i = share; i < s.count; i += 64) {
            f4 q;
            __builtin_memcpy(&q, s.part + i * p.N + at.at, 16);
            v[0] += q[0], v[1] += q[1], v[2] += q[2], v[3] += q[3];
        }
    } else if (at.any()) {
        for (int64_t i = share; i < s.count; i += 64)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < at.left) v[q] += s.part[i * p.N + at.at + q];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) sums[share][own * 4 + q] = v[q];
    const int row = threadIdx.x >> 6, col = threadIdx.x & 63;
    for (int o = 32; o >= 16; o >>= 1) {
        __syncthreads();
        for (int r = row; r < o; r += 16) sums[r][col] += sums[r + o][col];
    }
    for (int o = 8; o; o >>= 1) {
        __syncthreads();
        if (row < o) sums[row][col] += sums[row + o][col];
    }
    if (row == 0 && blockIdx.x * 64 + col < p.N) s.out[blockIdx.x * 64 + col] = sums[0][col];
}

__global__ __launch_bounds__(256) void zero_kernel(float *out, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) out[i] = 0.0f;
}

template <int DT, int WT, int TPR, int C, int MODE>
hipError_t run(const BlockNormArgs &a, hipStream_t s) {
    constexpr int ROWS = threads_of(TPR) / TPR;
    const int64_t blocks = (a.M + ROWS - 1) / ROWS, most = 256 * (2048 / threads_of(TPR));
    const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(threads_of(TPR));
    if (a.layer || a.post_bias || a.pre_bias) block_norm_kernel<DT, WT, TPR, C, MODE, true><<<grid, block, 0, s>>>(a);
    else block_norm_kernel<DT, WT, TPR, C, MODE, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

// The sums over no rows.  (a.gate_rows: the number of gates.)
hipError_t zero_sums(const BlockNormBackwardArgs &a, hipStream_t s) {
    float *const outs[5] = {a.dpre, a.dpre_bias, a.dpost, a.dpost_bias, a.dgate};
    for (int q = 0; q < 5; ++q) {
        if (!outs[q]) continue;
        const int64_t n = q < 4 ? a.N : a.gate_rows * a.N, blocks = (n + 255) / 256, most = (int64_t)1 << 20;
        zero_kernel<<<dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, s>>>(outs[q], n);
    }
    return hipGetLastError();
}

// Threads and pieces of a row: N <= 16384.
template <int DT, int MODE, typename F>
hipError_t sized(int N, F &&f) {
    using std::integral_constant;
    const int pieces = (N + kPiece<DT> - 1) / kPiece<DT>;
    auto call = [&](auto threads, auto each) { return f(threads, each); };
    if (pieces <= 64) return call(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if constexpr (MODE != kShort) {
        if (pieces <= 128) return call(integral_constant<int, 128>{}, integral_constant<int, 1>{});
        if (pieces <= 256) return call(integral_constant<int, 256>{}, integral_constant<int, 1>{});
        if (pieces <= 512) return call(integral_constant<int, 512>{}, integral_constant<int, 1>{});
        if (pieces <= 1024) return call(integral_constant<int, 512>{}, integral_constant<int, 2>{});
        if (pieces <= 2048) return call(integral_constant<int, 512>{}, integral_constant<int, 4>{});
        if constexpr (DT == kF32) return call(integral_constant<int, 512>{}, integral_constant<int, 8>{});
    }
    return hipErrorInvalidValue;
}

template <int DT, typename F>
hipError_t moded(int N, F &&f) {
    using std::integral_constant;
    constexpr int V = kPiece<DT>;
    if (N % V == 0) return sized<DT, kWhole>(N, [&](auto t, auto c) { return f(t, c, integral_constant<int, kWhole>{}); });
    if (N > V) return sized<DT, kTail>(N, [&](auto t, auto c) { return f(t, c, integral_constant<int, kTail>{}); });
    return sized<DT, kShort>(N, [&](auto t, auto c) { return f(t, c, integral_constant<int, kShort>{}); });
}

template <int DT, int WT, int TPR, int C, int MODE>
hipError_t run_back(const BlockNormBackwardArgs &a, hipStream_t s) {
    const Shares d = shares_of(a.M, a.N, a.M / a.gate_rows, DT);
    const dim3 grid((unsigned)d.workers), block(TPR);
    // (a bias's gradient may be asked for without its bias)
    const bool full = a.layer || a.post_bias || a.pre_bias || a.dpost_bias || a.dpre_bias;
    if (full) block_norm_backward_kernel<DT, WT, TPR, C, MODE, true><<<grid, block, 0, s>>>(a, d);
    else block_norm_backward_kernel<DT, WT, TPR, C, MODE, false><<<grid, block, 0, s>>>(a, d);
    return hipGetLastError();
}

template <int DT, int WT>
hipError_t forward(const BlockNormArgs &a, hipStream_t s) {
    return moded<DT>(a.N, [&](auto t, auto c, auto m) {
        return run<DT, WT, decltype(t)::value, decltype(c)::value, decltype(m)::value>(a, s);
    });
}

template <int DT, int WT>
hipError_t backward(const BlockNormBackwardArgs &a, hipStream_t s) {
    return moded<DT>(a.N, [&](auto t, auto c, auto m) {
        return run_back<DT, WT, decltype(t)::value, decltype(c)::value, decltype(m)::value>(a, s);
    });
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs &a, int dtype, bool wide_weights, hipStream_t s) {
    if (dtype == kF32) return forward<kF32, kF32>(a, s);
    if (dtype == kF16) return wide_weights ? forward<kF16, kF32>(a, s) : forward<kF16, kF16>(a, s);
    return wide_weights ? forward<kBF16, kF32>(a, s) : forward<kBF16, kBF16>(a, s);
}

size_t block_norm_backward_workspace(int64_t M, int64_t N, int64_t R, int dtype) {
    if (M == 0) return 0;
    const Shares d = shares_of(M, N, R, dtype);
    return (size_t)((4 * d.workers + (d.parts > 1 ? d.groups * d.parts : 0)) * N) * 4;
}

hipError_t launch_block_norm_backward(const BlockNormBackwardArgs &all, int dtype, bool wide_weights, void *ws, hipStream_t s) {
    BlockNormBackwardArgs a = all;
    a.part = static_cast<float *>(ws);
    hipError_t e = hipSuccess;
    if (a.M == 0) return zero_sums(a, s);
    if (dtype == kF32) e = backward<kF32, kF32>(a, s);
    else if (dtype == kF16) e = wide_weights ? backward<kF16, kF32>(a, s) : backward<kF16, kF16>(a, s);
    else e = wide_weights ? backward<kBF16, kF32>(a, s) : backward<kBF16, kBF16>(a, s);
    if (e != hipSuccess) return e;
    const int64_t R = a.M / a.gate_rows;
    const Shares d = shares_of(a.M, a.N, R, dtype);
    const bool gates = a.dgate && d.parts > 1;
    if (!a.dpre && !a.dpre_bias && !a.dpost && !a.dpost_bias && !gates) return e;
    PartSums p{};
    float *const outs[4] = {a.dpre, a.dpre_bias, a.dpost, a.dpost_bias};
    for (int q = 0; q < 4; ++q) p.s[q] = PartSum{a.part + q * d.workers * a.N, outs[q], d.workers};
    p.gate_part = a.part + 4 * d.workers * a.N, p.dgate = a.dgate, p.gate_parts = d.parts, p.N = a.N;
    block_norm_parts_kernel<<<dim3((unsigned)((a.N + 63) / 64), (unsigned)(4 + (gates ? R : 0))), dim3(1024), 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace tq2
