// A whole mixture-of-experts layer: norm, router, experts, residual.
#pragma once

#include "q4.h"

namespace tq2 {

struct LayerArgs {
    const void *x, *norm, *router;   // norm may be null
    bool wide_norm, wide_router;     // f32, else of x's type
    double eps;
    RouteArgs route;                 // its logits are the layer's own (f32)
    Q4View gate, up, down;
    const void *residual;            // may be null
    void *y;
    int64_t T;
    int dtype;
};

// Workspace: n [T][d] where there is a norm, the logits, then the experts' own.
struct LayerPlan {
    MoePlan moe;
    bool few;                        // two launches: the logits, and everything behind them
    size_t off_logits, off_moe, total;
};
// coarse: the weights' groups are of kFewGroup (the sizes do not depend on it, nor on the router's groups)
LayerPlan layer_plan(int64_t T, int64_t k, int64_t E, int64_t groups, int64_t d, int64_t f, int dtype, bool norm, bool coarse);
hipError_t launch_moe_layer(const LayerPlan &p, const LayerArgs &a, void *ws, int patience, hipStream_t s);

// moe_few.hip: the experts' choice and products of a few tokens, from their logits, in one launch, for weights in groups of kFewGroup.
struct FewArgs {
    const void *n;                   // [T][d], normed
    const float *logits;             // [T][E]
    void *h;                         // silu(g) u in bfloat16 parts [T k][parts][whole units of 128 from f], filled with bytes
                                     // of 0xff up to f and of 0 past it
    int patience;                    // how often a value is looked for before a workgroup forms it itself
};
hipError_t launch_few_experts(const FewArgs &f, const LayerArgs &a, hipStream_t s);
constexpr int kFewOwn = 4;           // experts of a lane that its router holds
constexpr int kFewGroup = 128;

}  // namespace tq2
