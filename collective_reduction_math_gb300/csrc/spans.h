// spans.h -- the memory that a call's arguments cover, and the check that no
// two of them overlap in a form that the call does not allow.  Host only.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "mr.h"
#include "mr_internal.h"

namespace mr {

// A byte range of the call, or (ld > 0) rows of `width` bytes every `ld` bytes from lo.
struct Span {
    uintptr_t lo, hi;
    size_t ld, width;
    const char* name;
    int rank;       // -1: not a rank buffer
    bool written;
};

// Room for kMost ranges; the caller adds no more.
template <int kMost>
struct Spans {
    Span s[kMost];
    int open[kMost];
    int n = 0;
    void add(const void* p, size_t bytes, const char* name, bool written) {
        if (p && bytes) s[n++] = {(uintptr_t)p, (uintptr_t)p + bytes, 0, 0, name, -1, written};
    }
    void add_rows(const void* p, size_t rows, size_t ld, size_t width, const char* name, int rank, bool written) {
        if (width) s[n++] = {(uintptr_t)p, (uintptr_t)p + (rows - 1) * ld + width, ld, width, name, rank, written};
    }
};

// Whether two overlapping ranges never share a byte: rows of one stride whose
// columns lie beside each other (column slices of one buffer).
inline bool beside(const Span& a, const Span& b) {
    if (!a.ld || a.ld != b.ld) return false;
    const Span &x = a.lo <= b.lo ? a : b, &y = a.lo <= b.lo ? b : a;
    const size_t d = (y.lo - x.lo) % x.ld;      // where y's columns start within x's rows
    return d >= x.width && d + y.width <= x.ld;
}

// `open`: room for n indexes.
inline mr_status_t check_spans(Span* s, int* open, int n) {
    const auto before = [](const Span& a, const Span& b) { return a.lo < b.lo; };
    if (!std::is_sorted(s, s + n, before)) std::sort(s, s + n, before);
    int nopen = 0;
    for (int i = 0; i < n; ++i) {
        const Span& b = s[i];
        int keep = 0;
        for (int j = 0; j < nopen; ++j) {
            const Span& a = s[open[j]];
            if (a.hi <= b.lo) continue;
            open[keep++] = open[j];
            if (!a.written && !b.written) continue;
            // in place: what a rank writes over its own input, row by row
            const bool in_place = a.rank >= 0 && a.rank == b.rank && a.written != b.written && a.lo == b.lo && a.ld == b.ld;
            if (!in_place && !beside(a, b))
                return report_error(MR_ERR_ALIAS, "%s[%d] overlaps %s[%d] in a form that is not an allowed in-place one",
                                    a.name, std::max(0, a.rank), b.name, std::max(0, b.rank));
        }
        nopen = keep;
        open[nopen++] = i;
    }
    return MR_OK;
}
template <int kMost>
mr_status_t check_spans(Spans<kMost>& v) {
    return check_spans(v.s, v.open, v.n);
}

inline bool misaligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

}  // namespace mr
