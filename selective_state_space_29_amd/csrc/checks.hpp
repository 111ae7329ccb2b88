// Argument checks that the entry points share: byte ranges and their overlaps, strides, workspaces.
#pragma once

#include <stdint.h>

#include "../../include/mamba_scan.h"

namespace mscan {

struct Bytes {
    uintptr_t lo = 0, hi = 0;
};

// Bytes of n0 rows, `s0` elements apart, of n1 rows, `s1` apart, of n2 elements of `es` bytes.
inline Bytes bytes_of(const void* p, int64_t es, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2) {
    Bytes b;
    if (!p || n0 <= 0 || n1 <= 0 || n2 <= 0) return b;
    b.lo = reinterpret_cast<uintptr_t>(p);
    b.hi = b.lo + (uintptr_t)(((n0 - 1) * s0 + (n1 - 1) * s1 + n2) * es);
    return b;
}
inline Bytes flat(const void* p, int64_t bytes) { return bytes_of(p, 1, 1, 0, 1, 0, bytes); }

inline bool meet(const Bytes& a, const Bytes& b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

template <int NI, int NO>
bool any_overlap(const Bytes (&ins)[NI], const Bytes (&outs)[NO]) {
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (meet(outs[o], ins[i])) return true;
        for (int o2 = 0; o2 < o; ++o2)
            if (meet(outs[o], outs[o2])) return true;
    }
    return false;
}

// Whether n rows `s` elements apart could not be addressed in 64 bits (or a size is negative).
inline bool bad_span(int64_t n, int64_t s) { return n < 0 || s < 0 || (n > 1 && s > ((int64_t)1 << 58) / n); }

inline bool bad_dtype(mamba_scan_dtype t) { return t != MAMBA_SCAN_F32 && t != MAMBA_SCAN_BF16; }
inline bool misaligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)a != 0; }

// A workspace of at least `need` bytes, 256-byte aligned.
inline int check_workspace(const void* ws, int64_t have, int64_t need) {
    if (have < 0 || (have > 0 && !ws)) return MAMBA_SCAN_ERR_ARGS;
    if (need > have) return MAMBA_SCAN_ERR_WORKSPACE;
    if (need > 0 && misaligned(ws, 256)) return MAMBA_SCAN_ERR_ARGS;
    return MAMBA_SCAN_OK;
}

constexpr int64_t kMaxGrid = 0x7fffffff;

}  // namespace mscan
