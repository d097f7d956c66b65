/*
 * libtq2 -- the parts of a transformer block around 4-bit weights, for AMD Instinct MI355X (gfx950):
 * a product with its bias, activation and residual, a whole mixture-of-experts layer, and the norms after and
 * before a block with its gate and residual scale, with their gradient.  The conventions are libtq2.h's and
 * libtq2_moe.h's: device pointers owned by the caller, `stream` a hipStream_t, calls asynchronous on it and acting on
 * the current device, status codes TQ2_E*, argument errors found on the host before anything is queued.
 */
#ifndef LIBTQ2_BLOCK_H
#define LIBTQ2_BLOCK_H

#include "libtq2_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { Q4_ACT_NONE = 0, Q4_ACT_RELU = 1, Q4_ACT_GELU = 2, Q4_ACT_GELU_TANH = 3, Q4_ACT_SILU = 4 };

/* y[m][n] = act(sum_k x[m][k] * W[n][k] + bias[n]) + residual[m][n] for a weight with E == 1: q4_gemm with its
 * epilogue in f32, rounded once.  bias [N] of type bias_dtype, which is Q4_F32 or dtype (NULL: none); residual [M][N] of type
 * dtype (NULL: none).  GELU is v Phi(v), GELU_TANH its form with tanh, SILU v / (1 + e^-v); all three are 0 at -infinity.
 * y may be the residual itself, and overlaps nothing else; the rest, the workspace
 * (q4_gemm_workspace_size bytes) included, is as for q4_gemm. */
int q4_linear(const q4_weight *w, const void *x, const void *bias, int bias_dtype, int activation, const void *residual,
              void *y, int64_t M, int dtype, void *workspace, size_t workspace_bytes, void *stream);

/* A whole mixture-of-experts layer on rows x [T][d]:
 *   n       = x / sqrt(mean(x^2) + eps) * norm, rounded to f32 and then to x's type (n = x without norm)
 *   logits  = n router^T, summed in f64 and rounded to f32
 *   idx, weights = moe_route's of those logits (its bias, groups, keep, group_top, score and renorm, its masks and ties)
 *   y[t]    = residual[t] + sum_j weights[t][j] * down_e(silu(gate_e n_t) * (up_e n_t)), e = idx[t][j]
 * x, residual and y [T][d] of type dtype; norm [d] of norm_dtype and router [E][d] of router_dtype, each Q4_F32 or dtype;
 * norm, bias and residual may be NULL.  gate, up and down, T and k as for q4_moe, k <= E, and with a norm d <= 16384; the
 * router's arguments as for moe_route.  idx and weights are written.  x, router, y and residual are 16-byte aligned.  y may be
 * the residual itself; beside that the outputs overlap neither each other nor the inputs. */
typedef struct moe_layer_call {
    const void *x, *norm, *router;
    const float *bias;
    const q4_weight *gate, *up, *down;
    const void *residual;
    void *y;
    int32_t *idx;
    float *weights;
    double eps;
    int64_t T, k, groups, keep, group_top;
    int32_t score, renorm, dtype, norm_dtype, router_dtype;
    int32_t reserved;
} moe_layer_call;

/* Bytes of device workspace that moe_layer needs (0 on bad sizes).  with_norm: the call has a norm. */
size_t moe_layer_workspace_size(int64_t T, int64_t k, int64_t E, int64_t d, int64_t f, int dtype, int with_norm);

/* workspace: moe_layer_workspace_size bytes, 256-byte aligned, clear of all else; its contents are scratch, and calls that
 * share one must not overlap in time.  Results are deterministic.  T == 0 is a no-op. */
int moe_layer(const moe_layer_call *call, void *workspace, size_t workspace_bytes, void *stream);

/* Test hook: with a few tokens, how often a workgroup looks for a value that another one forms before it forms it itself (the
 * results are the same bits), 0 to 65536, which it is at first: some tens of milliseconds.  Of the whole process.  Returns the old
 * setting, or TQ2_EINVAL. */
int moe_layer_set_patience(int tries);

/* The norms after and before a block, with its gate and residual scale:
 *   u = norm(b) * post + post_bias       (b itself without post)
 *   y = x + scale * gate * u, rounded to its type      (x itself without b)
 *   n = norm(y) * pre + pre_bias         (not formed without pre)
 * norm(v) = v / sqrt(mean(v^2) + eps), or with `layer` (v - mean(v)) / sqrt(var(v) + eps), over the N columns; statistics are
 * f64's.  x, b, y, n [M][N] of type dtype; post, post_bias, pre, pre_bias [N] and gate [R][N], all of weights_dtype, which is Q4_F32
 * or dtype; row m has gate row m / (M / R), R divides M.  Any pointer but x may be NULL: gate, post
 * and y belong to b, post_bias to post, pre_bias and n to pre; R is 1 without a gate.  y may be NULL where pre is given.
 * 1 <= N <= 16384; M == 0 is a no-op, M < 2^31.  Pointers are aligned to their elements; outputs overlap neither each other nor
 * inputs. */
typedef struct block_norm_call {
    const void *x, *b, *post, *post_bias, *gate, *pre, *pre_bias;
    void *y, *n;
    double eps;
    int64_t M, N, R;
    float scale;
    int32_t layer, dtype, weights_dtype;
} block_norm_call;
int block_norm(const block_norm_call *call, void *stream);

/* Gradient of block_norm: with dy and dn those of y and n,
 *   dx = dy + (gradient of dn through the second norm),  db = scale * gate * dx (through the first norm, with post),
 *   dgate = scale * sum of u * dx over a gate's rows, dpost, dpost_bias, dpre, dpre_bias the sums over all rows.
 * dy, dn, dx, db [M][N] of type dtype, the others f32: dgate [R][N], the rest [N]; all are overwritten.  Inputs as block_norm's, with y the
 * rows that it gave (x where there is no b).  dy may be NULL (0); dn and y go with pre; without pre they are NULL.  Outputs that are NULL are not
 * formed; db, dgate, dpost and dpost_bias need b, and what their names say.  f32 sums, whose order is fixed: results are
 * deterministic; sums over no rows are 0.  (A row's sum of dn * pre * y, and where there are means of y and of b, over the up to 32
 * columns of a thread, is one of them: where it passes f32's range, the row's gradient is not finite.)  A bias's gradient needs no
 * bias.  Outputs overlap neither each other nor inputs. */
typedef struct block_norm_backward_call {
    const void *dy, *dn, *y, *b, *post, *post_bias, *gate, *pre, *pre_bias;
    void *dx, *db;
    float *dgate, *dpost, *dpost_bias, *dpre, *dpre_bias;
    double eps;
    int64_t M, N, R;
    float scale;
    int32_t layer, dtype, weights_dtype;
} block_norm_backward_call;

/* Bytes of device workspace that block_norm_backward needs (0 on bad sizes, or for M == 0). */
size_t block_norm_backward_workspace_size(int64_t M, int64_t N, int64_t R, int dtype);
int block_norm_backward(const block_norm_backward_call *call, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBTQ2_BLOCK_H */
