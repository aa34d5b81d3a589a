// tb_host.h -- argument checks shared by the entry points of libtb.so (host code).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cmath>

#include "tb.h"

namespace tbh {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

struct Range {
    uintptr_t lo, hi;
};
inline Range range_of(const void *p, size_t bytes) { return {(uintptr_t)p, (uintptr_t)p + bytes}; }
inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// dq of a block is amax times this
inline float dq_unit() { return static_cast<float>(1.0 / (127.0 * std::sqrt(128.0))); }

// bytes of one element of a tb_dtype; 0 for an unknown one
inline size_t dtype_bytes(int t) { return t == TB_F32 ? 4 : t == TB_BF16 || t == TB_F16 ? 2 : 0; }

// One array argument of a call: where it lies, and whether the call writes it.
struct Arg {
    const void *p;
    size_t bytes;
    bool out;
};
// TB_EINVAL for a null array or for an output that overlaps any other array, TB_EALIGN for a
// misaligned one. `optional` arrays that are null are left out by the caller.
template <size_t N>
inline int check_args(const Arg (&a)[N], size_t n = N)
{
    for (size_t i = 0; i < n; ++i)
        if (!a[i].p)
            return TB_EINVAL;
    for (size_t i = 0; i < n; ++i)
        if (!aligned16(a[i].p))
            return TB_EALIGN;
    for (size_t i = 0; i < n; ++i)
        for (size_t j = 0; j < i; ++j)
            if ((a[i].out || a[j].out) && overlaps(range_of(a[i].p, a[i].bytes), range_of(a[j].p, a[j].bytes)))
                return TB_EINVAL;
    return TB_OK;
}

}  // namespace tbh
