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
    size_t off_logits, off_moe, total;
};
LayerPlan layer_plan(int64_t T, int64_t k, int64_t E, int64_t d, int64_t f, int dtype, bool norm);
hipError_t launch_moe_layer(const LayerPlan &p, const LayerArgs &a, void *ws, hipStream_t s);

}  // namespace tq2
