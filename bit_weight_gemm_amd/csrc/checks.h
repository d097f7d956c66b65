// Argument checks shared by the C entry points (host code).
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "../../include/libtq2_block.h"
#include "q4.h"

namespace tq2 {
namespace check {

inline bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

inline size_t size_of(int dtype) { return dtype == Q4_F32 ? 4 : 2; }

inline bool known(int dtype) { return dtype == Q4_F32 || dtype == Q4_F16 || dtype == Q4_BF16; }

inline bool weight_ok(const q4_weight *w) {
    return w && w->data && aligned(w->data, 256) && (w->zeros == 0 || w->zeros == 1) &&
           q4_packed_size(w->E, w->N, w->K, w->G, w->zeros) != 0;
}

inline Q4View view(const q4_weight *w) { return q4_view(w->data, w->E, w->N, w->K, w->G, w->zeros != 0); }

inline size_t bytes(const q4_weight *w) { return q4_packed_size(w->E, w->N, w->K, w->G, w->zeros); }

struct Range {
    const void *at;
    size_t bytes;
};

// A caller's workspace: large enough, 256-byte aligned, clear of the call's other arguments.
inline bool workspace_bad(const void *ws, size_t ws_bytes, size_t need, std::initializer_list<Range> others) {
    if (!ws || ws_bytes < need || !aligned(ws, 256)) return true;
    for (const Range &r : others)
        if (overlap(ws, need, r.at, r.bytes)) return true;
    return false;
}

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;

}  // namespace check
}  // namespace tq2
