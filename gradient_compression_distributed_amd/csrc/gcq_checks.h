// gcq_checks.h -- host-side argument checks shared by the files that define
// the C ABI (gcq_api.hip, gcq_api_lm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "gcq.h"

namespace gcq {
namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

struct Range {
    uintptr_t lo, hi;
    bool writable;
};

Range range(const void *p, size_t bytes, bool writable)
{
    return Range{(uintptr_t)p, (uintptr_t)p + bytes, writable};
}

// True when a writable range intersects any other range.  Sorted sweep:
// a pair (A before B in start order) overlaps iff B.lo < A.hi, so it is
// enough to track the largest end so far among writable and among all
// ranges.  Read-only ranges may overlap one another.
bool any_write_overlap(Range *first, Range *last)
{
    std::sort(first, last, [](const Range &a, const Range &b) { return a.lo < b.lo; });
    uintptr_t end_all = 0, end_w = 0;
    for (const Range *p = first; p != last; ++p) {
        const Range &r = *p;
        if (r.hi == r.lo)
            continue;
        if (r.lo < end_w || (r.writable && r.lo < end_all))
            return true;
        end_all = std::max(end_all, r.hi);
        if (r.writable)
            end_w = std::max(end_w, r.hi);
    }
    return false;
}

int launch_status(hipError_t e)
{
    if (e == hipSuccess)
        return GCQ_OK;
    if (e == hipErrorOutOfMemory)
        return GCQ_ERR_NOMEM;
    return GCQ_ERR_LAUNCH;
}

}  // namespace
}  // namespace gcq
