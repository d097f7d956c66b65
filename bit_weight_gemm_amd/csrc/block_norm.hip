// The norms after and before a block, with its gate and residual scale, and their gradient:
//   u = norm(b) post + post_bias (b itself without post)
//   y = x + scale gate u, rounded to its type
//   n = norm(y) pre + pre_bias
// with norm(v) = v / sqrt(mean(v^2) + eps), or (v - mean) / sqrt(var + eps).
//
// One pass over memory: TPR threads hold a row (C pieces of 16 bytes each), every input is read once, sums go over the
// wave by lane exchanges and over the waves through LDS.
#include "block_norm.h"

namespace tq2 {

namespace {

// Threads of a workgroup: rows of up to 256 threads share workgroups of 256.
constexpr int threads_of(int tpr) { return tpr < 256 ? 256 : tpr; }

// FULL: with means or biases.  The rows go round the workgroups.  Parameters that are the same for all rows stay in registers, and the next row's pieces are on
// their way while one is normed.
template <int DT, int WT, int TPR, int C, int MODE, bool FULL>
__global__ __launch_bounds__(threads_of(TPR)) void block_norm_kernel(BlockNormArgs p) {
    constexpr int V = kPiece<DT>, ROWS = threads_of(TPR) / TPR;
    constexpr bool HOLD = C == 1;  // (two pieces and more of everything would not fit)
    __shared__ double room[2][TPR / 64 * 2];
    const int tid = threadIdx.x % TPR, N = p.N;
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
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
        return norm_of(sum[1], sum[0], N, p.layer, p.eps);
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
// The sums over rows are kept in f32 by the workgroup that has the rows, in registers, and written as one part each;
// a second kernel adds the parts in their order.

// Workgroups: `parts` to each run of rows that share a gate, or whole runs to a workgroup.
struct Shares {
    int64_t groups, parts;   // runs of rows with one gate; workgroups of a run (1: whole runs, dealt round)
    int64_t workers;         // workgroups
};
constexpr int64_t kWorkers = 256;
Shares shares_of(int64_t M, int64_t R) {
    Shares s;
    s.groups = R;
    const int64_t run = M / R;
    s.parts = R >= kWorkers ? 1 : kWorkers / R;
    if (s.parts > run) s.parts = run;
    s.workers = s.parts > 1 || R <= kWorkers ? R * s.parts : kWorkers;
    return s;
}

template <int DT, int WT, int TPR, int C, int MODE>
__global__ __launch_bounds__(TPR) void block_norm_backward_kernel(BlockNormBackwardArgs p, Shares s) {
    constexpr int V = kPiece<DT>;
    __shared__ double wide[TPR / 64 * 4];
    __shared__ float room[2][TPR / 64 * 2];
    const int tid = threadIdx.x, N = p.N;
    float dpre[C][V] = {}, dpre_bias[C][V] = {}, dpost[C][V] = {}, dpost_bias[C][V] = {};
    const int64_t run = p.gate_rows;
    for (int64_t job = blockIdx.x; job < s.groups * s.parts; job += gridDim.x) {
        const int64_t group = job / s.parts, part = job % s.parts;
        const int64_t r0 = group * run + run * part / s.parts, r1 = group * run + run * (part + 1) / s.parts;
        float dgate[C][V] = {};
        for (int64_t row = r0; row < r1; ++row) {
            const int64_t at = row * N;
            Raw<DT, V> ry[C], rb[C], rdy[C], rdn[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const Piece<V, MODE> q(tid + TPR * c, N);
                if (p.pre) q.template load<DT>(p.y, at, N, ry[c]), q.template load<DT>(p.dn, at, N, rdn[c]);
                if (p.b) q.template load<DT>(p.b, at, N, rb[c]);
                if (p.dy) q.template load<DT>(p.dy, at, N, rdy[c]);
            }
            float y[C][V], b[C][V], d[C][V];
            double sum[4] = {};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const Piece<V, MODE> q(tid + TPR * c, N);
                if (p.pre) {
                    q.template values<DT>(ry[c], y[c]);
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[0] += y[c][i], sum[1] += (double)y[c][i] * y[c][i];
                }
                if (p.b) {
                    q.template values<DT>(rb[c], b[c]);
                    if (p.post) {
#pragma unroll
                        for (int i = 0; i < V; ++i) sum[2] += b[c][i], sum[3] += (double)b[c][i] * b[c][i];
                    }
                }
                if (p.dy) {
                    q.template values<DT>(rdy[c], d[c]);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) d[c][i] = 0.0f;
                }
            }
            row_total<TPR, 4>(sum, wide);
            if (p.pre) {
                const Norm r = norm_of(sum[0], sum[1], N, p.layer, p.eps);
                const float rstd = (float)r.rstd;
                float g[C][V], gs[2] = {};
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const Piece<V, MODE> q(tid + TPR * c, N);
                    float dn[V], w[V];
                    Raw<WT, V> rw;
                    q.template load<WT>(p.pre, 0, N, rw);
                    q.template values<WT>(rw, w);
                    q.template values<DT>(rdn[c], dn);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        y[c][i] = (float)((double)y[c][i] - r.mean) * rstd;
                        g[c][i] = dn[i] * w[i];
                        gs[0] += g[c][i], gs[1] += g[c][i] * y[c][i];
                        dpre[c][i] += dn[i] * y[c][i], dpre_bias[c][i] += dn[i];
                    }
                    // (past the row's end y^ is -mean rstd, but dn and w are 0)
                }
                row_total<TPR, 2>(gs, room[0]);
                const float m0 = p.layer ? gs[0] / N : 0.0f, m1 = gs[1] / N;
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < V; ++i) d[c][i] += (g[c][i] - m0 - y[c][i] * m1) * rstd;
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (p.dx) Piece<V, MODE>(tid + TPR * c, N).template store<DT>(p.dx, at, d[c]);
            if (!p.b) {
                if constexpr (TPR > 64) __syncthreads();
                continue;
            }
            const int64_t gate_at = p.gate ? group * N : 0;
            if (p.post) {
                const Norm r = norm_of(sum[2], sum[3], N, p.layer, p.eps);
                const float rstd = (float)r.rstd;
                float gs[2] = {};
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const Piece<V, MODE> q(tid + TPR * c, N);
                    float w[V], k[V] = {}, gate[V];
                    Raw<WT, V> rw;
                    q.template load<WT>(p.post, 0, N, rw);
                    q.template values<WT>(rw, w);
                    if (p.post_bias) q.template load<WT>(p.post_bias, 0, N, rw), q.template values<WT>(rw, k);
                    if (p.gate) q.template load<WT>(p.gate, gate_at, N, rw), q.template values<WT>(rw, gate);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float hat = (float)((double)b[c][i] - r.mean) * rstd;
                        const float live = !q.any() || (MODE != kWhole && i >= q.left) ? 0.0f : d[c][i];
                        dgate[c][i] += (hat * w[i] + k[i]) * live;
                        const float du = p.scale * (p.gate ? gate[i] : 1.0f) * live;
                        dpost[c][i] += du * hat, dpost_bias[c][i] += du;
                        b[c][i] = hat;
                        d[c][i] = du * w[i];
                        gs[0] += d[c][i], gs[1] += d[c][i] * hat;
                    }
                }
                row_total<TPR, 2>(gs, room[1]);
                const float m0 = p.layer ? gs[0] / N : 0.0f, m1 = gs[1] / N;
#pragma unroll
                for (int c = 0; c < C; ++c) {
#pragma unroll
                    for (int i = 0; i < V; ++i) d[c][i] = (d[c][i] - m0 - b[c][i] * m1) * rstd;
                }
            } else {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const Piece<V, MODE> q(tid + TPR * c, N);
                    float gate[V];
                    Raw<WT, V> rw;
                    if (p.gate) q.template load<WT>(p.gate, gate_at, N, rw), q.template values<WT>(rw, gate);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        dgate[c][i] += b[c][i] * d[c][i];
                        d[c][i] *= p.scale * (p.gate ? gate[i] : 1.0f);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (p.db) Piece<V, MODE>(tid + TPR * c, N).template store<DT>(p.db, at, d[c]);
            if constexpr (TPR > 64) __syncthreads();  // the sums' rooms are free again
        }
        if (p.dgate) {  // scaled here: the parts are sums of finished terms
#pragma unroll
            for (int c = 0; c < C; ++c) {
#pragma unroll
                for (int i = 0; i < V; ++i) dgate[c][i] *= p.scale;
                float *out = s.parts == 1 ? p.dgate : p.part + (int64_t)gridDim.x * 4 * N;
                // V floats are more than a piece of f32 where the rows have 16 bits
                const int col = (tid + TPR * c) * V;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (col + i < N) out[job * N + col + i] = dgate[c][i];
            }
        }
    }
    auto put = [&](bool asked, int which, const float (&v)[C][V]) {
        if (!asked) return;
        float *out = p.part + ((int64_t)which * gridDim.x + blockIdx.x) * N;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (tid + TPR * c) * V;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (col + i < N) out[col + i] = v[c][i];
        }
    };
    put(p.dpre, 0, dpre), put(p.dpre_bias, 1, dpre_bias), put(p.dpost, 2, dpost), put(p.dpost_bias, 3, dpost_bias);
}

// out[which][n] = the sum of `count` parts, in an order that depends on their number alone: sixteen threads of a column
// take every sixteenth each, and their sums are added in pairs.
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
    __shared__ float sums[16][64];
    const int col = blockIdx.x * 64 + (threadIdx.x & 63), share = threadIdx.x >> 6;
    PartSum s;
    if (blockIdx.y < 4) s = p.s[blockIdx.y];
    else s = PartSum{p.gate_part + (int64_t)(blockIdx.y - 4) * p.gate_parts * p.N, p.dgate + (int64_t)(blockIdx.y - 4) * p.N,
                     p.gate_parts};
    if (!s.out) return;  // the whole workgroup
    float v = 0.0f;
    if (col < p.N)
        for (int64_t i = share; i < s.count; i += 16) v += s.part[i * p.N + col];
    sums[share][threadIdx.x & 63] = v;
    for (int o = 8; o; o >>= 1) {
        __syncthreads();
        if (share < o) sums[share][threadIdx.x & 63] += sums[share + o][threadIdx.x & 63];
    }
    if (share == 0 && col < p.N) s.out[col] = sums[0][threadIdx.x];
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

// Threads and pieces of a row.
template <int DT, int WT, int MODE>
hipError_t sized(const BlockNormArgs &a, hipStream_t s) {
    const int pieces = (a.N + kPiece<DT> - 1) / kPiece<DT>;
    if (pieces <= 64) return run<DT, WT, 64, 1, MODE>(a, s);
    if constexpr (MODE != kShort) {
        if (pieces <= 256) return run<DT, WT, 256, 1, MODE>(a, s);
        if (pieces <= 512) return run<DT, WT, 512, 1, MODE>(a, s);
        if (pieces <= 1024) return run<DT, WT, 1024, 1, MODE>(a, s);
        if (pieces <= 2048) return run<DT, WT, 1024, 2, MODE>(a, s);
        if constexpr (DT == kF32) return run<DT, WT, 1024, 4, MODE>(a, s);  // N <= 16384
    }
    return hipErrorInvalidValue;
}

template <int DT, int WT>
hipError_t moded(const BlockNormArgs &a, hipStream_t s) {
    constexpr int V = kPiece<DT>;
    if (a.N % V == 0) return sized<DT, WT, kWhole>(a, s);
    return a.N > V ? sized<DT, WT, kTail>(a, s) : sized<DT, WT, kShort>(a, s);
}

template <int DT, int WT, int TPR, int C, int MODE>
hipError_t run_back(const BlockNormBackwardArgs &a, hipStream_t s) {
    const Shares d = shares_of(a.M, a.M / a.gate_rows);
    block_norm_backward_kernel<DT, WT, TPR, C, MODE><<<dim3((unsigned)d.workers), dim3(TPR), 0, s>>>(a, d);
    return hipGetLastError();
}

template <int DT, int WT, int MODE>
hipError_t sized_back(const BlockNormBackwardArgs &a, hipStream_t s) {
    const int pieces = (a.N + kPiece<DT> - 1) / kPiece<DT>;
    if (pieces <= 64) return run_back<DT, WT, 64, 1, MODE>(a, s);
    if constexpr (MODE != kShort) {
        if (pieces <= 256) return run_back<DT, WT, 256, 1, MODE>(a, s);
        if (pieces <= 512) return run_back<DT, WT, 512, 1, MODE>(a, s);
        if (pieces <= 1024) return run_back<DT, WT, 1024, 1, MODE>(a, s);
        if (pieces <= 2048) return run_back<DT, WT, 1024, 2, MODE>(a, s);
        if constexpr (DT == kF32) return run_back<DT, WT, 1024, 4, MODE>(a, s);  // N <= 16384
    }
    return hipErrorInvalidValue;
}

template <int DT, int WT>
hipError_t moded_back(const BlockNormBackwardArgs &a, hipStream_t s) {
    constexpr int V = kPiece<DT>;
    if (a.N % V == 0) return sized_back<DT, WT, kWhole>(a, s);
    return a.N > V ? sized_back<DT, WT, kTail>(a, s) : sized_back<DT, WT, kShort>(a, s);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs &a, int dtype, bool wide_weights, hipStream_t s) {
    if (dtype == kF32) return moded<kF32, kF32>(a, s);
    if (dtype == kF16) return wide_weights ? moded<kF16, kF32>(a, s) : moded<kF16, kF16>(a, s);
    return wide_weights ? moded<kBF16, kF32>(a, s) : moded<kBF16, kBF16>(a, s);
}

size_t block_norm_backward_workspace(int64_t M, int64_t N, int64_t R) {
    if (M == 0) return 0;
    const Shares d = shares_of(M, R);
    return (size_t)((4 * d.workers + (d.parts > 1 ? d.groups * d.parts : 0)) * N) * 4;
}

hipError_t launch_block_norm_backward(const BlockNormBackwardArgs &all, int dtype, bool wide_weights, void *ws, hipStream_t s) {
    BlockNormBackwardArgs a = all;
    a.part = static_cast<float *>(ws);
    hipError_t e = hipSuccess;
    if (a.M == 0) return zero_sums(a, s);
    if (dtype == kF32) e = moded_back<kF32, kF32>(a, s);
    else if (dtype == kF16) e = wide_weights ? moded_back<kF16, kF32>(a, s) : moded_back<kF16, kF16>(a, s);
    else e = wide_weights ? moded_back<kBF16, kF32>(a, s) : moded_back<kBF16, kBF16>(a, s);
    if (e != hipSuccess) return e;
    const int64_t R = a.M / a.gate_rows;
    const Shares d = shares_of(a.M, R);
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
