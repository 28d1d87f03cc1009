// ssd_checks.h -- host-side argument checks shared by the C ABI translation units.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace ssd {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The bytes [lo, hi) of an array; empty for a null pointer or zero bytes.
struct Range {
    uintptr_t lo = 0, hi = 0;
    Range() = default;
    Range(const void *p, size_t bytes)
        : lo(reinterpret_cast<uintptr_t>(p)), hi(reinterpret_cast<uintptr_t>(p) + (p ? bytes : 0)) {}
    bool overlaps(const Range &o) const { return lo < o.hi && o.lo < hi; }
    bool same(const Range &o) const { return lo == o.lo && hi == o.hi; }
};

// Whether any output overlaps an input or another output.
template <size_t NI, size_t NO>
inline bool any_alias(const Range (&ins)[NI], const Range (&outs)[NO]) {
    for (size_t i = 0; i < NO; ++i) {
        for (size_t j = 0; j < NI; ++j)
            if (outs[i].overlaps(ins[j])) return true;
        for (size_t j = i + 1; j < NO; ++j)
            if (outs[i].overlaps(outs[j])) return true;
    }
    return false;
}

}  // namespace ssd
