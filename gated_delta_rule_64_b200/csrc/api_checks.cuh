// Argument checks shared by the C-ABI entry points (host code only).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "gdn_internal.cuh"

namespace gdn {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

struct Range {
    uintptr_t lo, hi;
};
inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
inline Range range_of(const void *p, size_t bytes) { return {(uintptr_t)p, (uintptr_t)p + bytes}; }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Sizes, head widths, dtype, gate kind (per head or per channel) and scale of a description.
gdn_status check_desc(const gdn_desc *d);
// Forgets the calling thread's last failure (every entry point begins with it).
void clear_error();

}  // namespace gdn
