// Rows held in the registers of one or more waves, as the norms work on them: sums over a row, packs of values
// at any place, and the choice of how many a lane takes.
#pragma once

#include <initializer_list>
#include <type_traits>
#include <utility>

#include "layers_common.hpp"

namespace mscan {

// Sums of N values over the WPR waves of a row, the same bits in every thread. `slot` alternates
// between calls, so one barrier a call is enough.
template <int N, int WPR, int WAVES>
__device__ __forceinline__ void row_sum(float (&v)[2], float (*lds)[2][WAVES], int slot, int wave) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) lds[slot][k][wave] = v[k];
        __syncthreads();
        const int first = wave / WPR * WPR;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < WPR; ++q) s += lds[slot][k][first + q];
            v[k] = s;
        }
    }
}

// n of V consecutive values (all of them in one access of any alignment), zeros behind them.
template <typename S, int V>
__device__ __forceinline__ Pack<S, V> load_some(const S* p, int n) {
    Pack<S, V> r{};
    if (n >= V) {
        __builtin_memcpy(&r, p, sizeof(r));
    } else if (n > 0) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < n) r.v[k] = p[k];
    }
    return r;
}
template <typename S, int V>
__device__ __forceinline__ void store_some(S* p, const Pack<S, V>& r, int n) {
    if (n >= V) {
        __builtin_memcpy(p, &r, sizeof(r));
    } else if (n > 0) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < n) p[k] = r.v[k];
    }
}

// The smallest instantiated number of packs that holds `nv` (1, 2, 3, 4, 6, 8, 12, 16, 24, 32; at most M).
template <int M, int N = 1, typename F>
auto with_packs(int64_t nv, F&& f) {
    constexpr int next = N < 4 ? N + 1 : N % 3 == 0 ? N / 3 * 4 : N / 2 * 3;
    if constexpr (next > M || N >= M) {
        return f(std::integral_constant<int, N < M ? M : N>{});
    } else {
        return nv <= N ? f(std::integral_constant<int, N>{}) : with_packs<M, next>(nv, f);
    }
}

// Entries q0 .. q1 - 1 of a column, `wide` apart, added in order, 16 loads on their way at a time.
__device__ __forceinline__ float column_sum(const float* part, int64_t wide, int64_t c, int q0, int q1) {
    float s = 0.0f;
    for (int q = q0; q < q1; q += 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = part[(int64_t)(q + i < q1 ? q + i : q1 - 1) * wide + c];
#pragma unroll
        for (int i = 0; i < 16; ++i) s += q + i < q1 ? v[i] : 0.0f;
    }
    return s;
}

// The widest pack (16 bytes and down) that the width, pointers and row strides are multiples of, and that
// leaves less than half of a wave idle over the width (200000 x 100 bf16: 141 us with packs of 4, on 25
// lanes, 113 with single elements).
template <typename S, int V = 16 / sizeof(S), typename F>
auto with_pack(int64_t dim, std::initializer_list<std::pair<const void*, int64_t>> rows, F&& f) {
    if constexpr (V == 1) {
        return f(std::integral_constant<int, 1>{});
    } else {
        bool ok = dim % V == 0 && dim > 32 * V;
        for (const auto& r : rows)
            ok = ok && (!r.first || (reinterpret_cast<uintptr_t>(r.first) % (V * sizeof(S)) == 0 && r.second % V == 0));
        return ok ? f(std::integral_constant<int, V>{}) : with_pack<S, V / 2>(dim, rows, f);
    }
}

}  // namespace mscan
