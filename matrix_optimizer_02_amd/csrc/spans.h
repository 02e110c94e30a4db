// Byte ranges of a call's buffers, for the check that no written one overlaps another.
#pragma once

#include <algorithm>
#include <cstdint>
#include <vector>

namespace dmuon {

// A caller buffer's byte range and whether the call writes it.
struct Span {
    uintptr_t lo, hi;
    bool written;
};

// True when no two of the spans overlap where one of them is written.  Read-
// only spans may overlap each other (the same gradient passed twice is
// harmless).  Sorted by start, a span overlaps an earlier one exactly when it
// starts below that one's end, so one sweep suffices.
inline bool disjoint_where_written(std::vector<Span>& v) {
    const auto before = [](const Span& x, const Span& y) { return x.lo < y.lo; };
    if (!std::is_sorted(v.begin(), v.end(), before)) std::sort(v.begin(), v.end(), before);
    uintptr_t end_any = 0, end_written = 0;
    for (const Span& sp : v) {
        if (sp.lo < end_written || (sp.written && sp.lo < end_any)) return false;
        end_any = std::max(end_any, sp.hi);
        if (sp.written) end_written = std::max(end_written, sp.hi);
    }
    return true;
}

}  // namespace dmuon
