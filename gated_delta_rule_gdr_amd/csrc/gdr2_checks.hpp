// gdr2_checks.hpp -- host-side argument checks shared by the C-ABI sources.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace {

struct Range {
    const void* p;
    size_t n;
};

inline bool overlap(const Range& a, const Range& b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline bool dims_ok(int64_t d) { return d == 64 || d == 128; }

// Any output overlapping any input or another output?
inline bool any_alias(const Range* outs, int no, const Range* ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// a * b <= lim for a, b >= 0, decided without forming a product that could overflow
inline bool prod_le(int64_t a, int64_t b, int64_t lim) { return a == 0 || b <= lim / a; }

}  // namespace
