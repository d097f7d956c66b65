/*
 * libtq2 -- 4-bit weights under group scales and mixture-of-experts operators for
 * AMD Instinct MI355X (gfx950).  The conventions are libtq2.h's: device pointers
 * owned by the caller, `stream` a hipStream_t (NULL: the legacy default stream),
 * calls asynchronous on it and acting on the current device, status codes TQ2_E*,
 * argument errors found on the host before anything is queued.
 */
#ifndef LIBTQ2_MOE_H
#define LIBTQ2_MOE_H

#include "libtq2.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { Q4_F32 = 0, Q4_F16 = 1, Q4_BF16 = 2 };                  /* types of activations, outputs and logits */
enum { MOE_SOFTMAX = 0, MOE_SIGMOID = 1 };                     /* router scores */

/* A packed 4-bit weight [E][N][K] in device memory that the caller owns: E experts
 * (1 for a dense weight), each W[n][k] = (code - zero) * scale, with one f16 scale and
 * one zero point per row and group of G consecutive k.  Filled in by the caller; `data`
 * is written by q4_pack. */
typedef struct q4_weight {
    void *data;        /* q4_packed_size bytes, 256-byte aligned */
    int64_t E, N, K, G;
    int32_t zeros;     /* 1: zero points were given, 0: all are 8 */
    int32_t reserved;
} q4_weight;

/* Bytes of a packed weight; 0 on bad sizes.  E, N >= 1; G is 32, 64 or 128; K a
 * multiple of G, K <= 2^20, and N <= 2^24; E <= 1024. */
size_t q4_packed_size(int64_t E, int64_t N, int64_t K, int64_t G, int zeros);

/* Packs codes u8 [E][N][K/2] (element 2j in the low four bits of byte j, 2j+1 in the
 * high ones; 4-byte aligned), scales f16 [E][N][K/G] and zeros u8 [E][N][K/G] (any byte;
 * NULL exactly when w->zeros is 0), all in device memory, into w->data.  Scales are taken
 * as they are: an infinite or NaN one gives such weights, and products with them are
 * infinite or NaN (which of the two may depend on the number of rows). */
int q4_pack(const q4_weight *w, const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros, void *stream);

/* w_out[e][n][k] = (code - zero) * scale as f32, exact. */
int q4_dequant(const q4_weight *w, float *w_out, void *stream);

/* Bytes of device workspace that q4_gemm needs for these sizes (0: none, as for up to
 * 32 rows; also 0 on bad sizes). */
size_t q4_gemm_workspace_size(const q4_weight *w, int64_t M, int dtype);

/* y[m][n] = sum_k x[m][k] * W[n][k] for a weight with E == 1.  x [M][K] and y [M][N]
 * have the type `dtype`, are row-major and 16-byte aligned and do not overlap; y is
 * overwritten, its values rounded once from f32 sums (nearest even).  Results are
 * deterministic.  M == 0 is a no-op; M < 2^31.  workspace: q4_gemm_workspace_size bytes,
 * 256-byte aligned, clear of x, y and the weight (NULL where that is 0); calls that share
 * one must not overlap in time. */
int q4_gemm(const q4_weight *w, const void *x, void *y, int64_t M, int dtype, void *workspace, size_t workspace_bytes,
            void *stream);

/* A mixture's router.  Per token t of T: scores p = softmax or sigmoid of logits
 * [T][E]; keys p + bias[e] (bias f32 [E] or NULL), or the logits themselves, which
 * order the same, where there is no bias and group_top or groups is 1.  The experts lie in `groups`
 * equal groups; a group's key is the sum of its group_top (1 or 2) largest keys, and the
 * experts of the `keep` best groups stay.  idx [T][k] (int32) are the experts with
 * the k largest keys, in that order, equal keys by the lower index; weights [T][k] (f32)
 * their scores, divided by their sum if renorm is not 0.  Keys are formed and compared
 * in f64.
 * A logit (or bias) of -inf masks its expert: it is never chosen, and slots that find
 * no expert get idx -1 and weight 0.  A NaN key ranks first.  A logit of NaN or +inf makes
 * every softmax score of its row NaN.
 * 1 <= E <= 1024, 1 <= k <= min(64, E), 1 <= groups <= 64, E % groups == 0,
 * 1 <= keep <= groups; logits, idx and weights aligned to their elements; outputs do
 * not overlap each other or the inputs.  T == 0 is a no-op; T < 2^31. */
int moe_route(const void *logits, const float *bias, int32_t *idx, float *weights, int64_t T, int64_t E, int64_t k,
              int64_t groups, int64_t keep, int64_t group_top, int score, int renorm, int dtype, void *stream);

/* Gradient of moe_route's weights with respect to the logits, the choice held fixed:
 * dlogits [T][E] (of the logits' type, overwritten) from dw = d(weights) f32 [T][k] and
 * the idx that moe_route gave (entries outside 0 .. E-1 have no weight and add nothing; an expert
 * that a row names twice gets both contributions).  f32 sums.  Renormalised, only
 * the chosen experts' logits have a gradient; where a row's scores (in f64) add up to 0, it is 0. */
int moe_route_backward(const void *logits, const int32_t *idx, const float *dw, void *dlogits, int64_t T, int64_t E,
                       int64_t k, int score, int renorm, int dtype, void *stream);

/* Bytes of device workspace that q4_moe needs (0 on bad sizes): T tokens of k slots, E
 * experts, gate and up [E][f][d], down [E][d][f]. */
size_t q4_moe_workspace_size(int64_t T, int64_t k, int64_t E, int64_t d, int64_t f, int dtype);

/* Experts' gated products: y[t] = sum_j weights[t][j] * down_e(silu(gate_e x_t) * (up_e x_t))
 * with e = idx[t][j]; slots whose idx is outside 0 .. E-1 are dropped (a token without
 * slots gets 0).  x and y [T][d] of type dtype; idx int32 [T][k], weights f32 [T][k];
 * gate and up [E][f][d] with equal G and both or neither with zero points, down [E][d][f].
 * Sums are f32, in an order that does not depend on timing: results are deterministic.
 * x and y 16-byte aligned, not overlapping; 1 <= k <= 64; T * k < 2^24; T == 0 is a no-op.
 * workspace: q4_moe_workspace_size bytes, 256-byte aligned, clear of all else; its contents are
 * scratch, and calls that share one must not overlap in time. */
int q4_moe(const void *x, const int32_t *idx, const float *weights, const q4_weight *gate, const q4_weight *up,
           const q4_weight *down, void *y, int64_t T, int64_t k, int dtype, void *workspace, size_t workspace_bytes,
           void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBTQ2_MOE_H */
