// A thread's piece of a row: 16 bytes or more, of any alignment that its elements have (gfx950).
#pragma once

#include <type_traits>

#include "q4.h"

namespace tq2 {

// ---- a thread's piece of a row: 16 bytes, V elements from column `at` on

template <int DT>
constexpr int kPiece = DT == kF32 ? 4 : 8;

// How a piece that does not lie within the row's N columns is read: kWhole: there is none but empty ones (N is a
// multiple of V); kTail: the last one is read up to the row's end and shifted (N >= V); kShort: element by element.
enum PieceMode { kWhole = 0, kTail = 1, kShort = 2 };

// V elements of type DT, any alignment of an element's.
template <int DT, int V>
struct Raw {
    w4 v[V * (DT == kF32 ? 4 : 2) / 16];
};
template <int DT, int V>
__device__ __forceinline__ void raw_values(const Raw<DT, V> &r, float (&out)[V]) {
#pragma unroll
    for (int q = 0; q < V; ++q) {
        if constexpr (DT == kF32) {
            const uint32_t b = r.v[q >> 2][q & 3];
            out[q] = __builtin_bit_cast(float, b);
        } else {
            const uint32_t w = r.v[q >> 3][(q >> 1) & 3];
            if constexpr (DT == kF16) out[q] = half_bits(q & 1 ? w >> 16 : w);
            else out[q] = __builtin_bit_cast(float, q & 1 ? w & 0xffff0000u : w << 16);
        }
    }
}

// The piece's place in a row of N columns.
template <int V, int MODE>
struct Piece {
    int at, left;  // first column; columns from there on (<= 0: none)
    __device__ Piece(int piece, int N) : at(piece * V), left(N - piece * V) {}
    __device__ bool full() const { return left >= V; }
    __device__ bool any() const { return left > 0; }

    template <int DT>
    __device__ __forceinline__ void load(const void *p, int64_t row, int N, Raw<DT, V> &r) const {
        constexpr int S = DT == kF32 ? 4 : 2;
        const char *b = static_cast<const char *>(p) + row * S;
        if constexpr (MODE == kShort) {
            r = Raw<DT, V>{};
#pragma unroll
            for (int q = 0; q < V; ++q)
                if (q < left) __builtin_memcpy(reinterpret_cast<char *>(&r) + q * S, b + (uint32_t)((at + q) * S), S);
        } else {
            const int from = full() ? at : MODE == kTail && any() ? N - V : 0;  // (none: the row's first, unused)
            __builtin_memcpy(&r, b + (uint32_t)(from * S), V * S);  // (unsigned: a scalar base and an offset of 32 bits)
        }
    }
    // The piece's values, zeros past the row's end.
    template <int DT>
    __device__ __forceinline__ void values(const Raw<DT, V> &r, float (&v)[V]) const {
        raw_values<DT, V>(r, v);
        if constexpr (MODE == kTail) {
            const int by = full() || !any() ? 0 : V - left;
#pragma unroll
            for (int o = 1; o < V; o <<= 1)
#pragma unroll
                for (int q = 0; q < V; ++q) v[q] = by & o ? (q + o < V ? v[q + o] : 0.0f) : v[q];
        }
        if constexpr (MODE != kShort) {
#pragma unroll
            for (int q = 0; q < V; ++q) v[q] = any() ? v[q] : 0.0f;
        }
    }
    // Rounds to nearest even.
    template <int DT>
    __device__ __forceinline__ void store(void *p, int64_t row, const float (&v)[V]) const {
        constexpr int S = DT == kF32 ? 4 : 2;
        using E = std::conditional_t<DT == kF32, float, std::conditional_t<DT == kF16, _Float16, __bf16>>;
        E e[V];
#pragma unroll
        for (int q = 0; q < V; ++q) e[q] = (E)v[q];
        char *b = static_cast<char *>(p) + row * S + (uint32_t)(at * S);
        if (full()) __builtin_memcpy(b, e, V * S);
        else if (MODE != kWhole)
#pragma unroll
            for (int q = 0; q < V; ++q)
                if (q < left) __builtin_memcpy(b + q * S, &e[q], S);
    }
};

}  // namespace tq2
