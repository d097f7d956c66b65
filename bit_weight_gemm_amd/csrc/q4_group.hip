// Launches of the experts' products with few rows each.
#include "q4_group.h"

namespace tq2 {

namespace {

template <int DT, int P>
hipError_t gate_up(const Q4GroupArgs &a, hipStream_t s) {
    if (a.w.G == 32) return run_q4_group<DT, P, 32, 2, 2, kGroupGateUp>(a, s);
    if (a.w.G == 64) return run_q4_group<DT, P, 64, 2, 2, kGroupGateUp>(a, s);
    return run_q4_group<DT, P, 128, 2, 2, kGroupGateUp>(a, s);
}

template <int P>
hipError_t down(const Q4GroupArgs &a, hipStream_t s) {
    if (a.w.G == 32) return run_q4_group<kF32, P, 32, 1, 4, kGroupDown>(a, s);
    if (a.w.G == 64) return run_q4_group<kF32, P, 64, 1, 4, kGroupDown>(a, s);
    return run_q4_group<kF32, P, 128, 1, 4, kGroupDown>(a, s);
}

}  // namespace

hipError_t launch_q4_group_gate_up(const Q4GroupArgs &a, int dtype, hipStream_t s) {
    if (dtype == kF32) return gate_up<kF32, 2>(a, s);
    if (dtype == kF16) return gate_up<kF16, 1>(a, s);
    return gate_up<kBF16, 1>(a, s);
}

hipError_t launch_q4_group_down(const Q4GroupArgs &a, int planes, hipStream_t s) {
    return planes == 1 ? down<1>(a, s) : down<2>(a, s);
}

}  // namespace tq2
