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

// Whether two overlapping ranges of a call are allowed: both are read, or a rank
// writes over its own input, row by row, or they share no byte.
inline bool allowed(const Span& a, const Span& b) {
    if (!a.written && !b.written) return true;
    return (a.rank >= 0 && a.rank == b.rank && a.written != b.written && a.lo == b.lo && a.ld == b.ld) || beside(a, b);
}

// `open`: room for n indexes.  In the order of their starts, each range meets
// those that have not ended: one that is read meets the written ones, which are few
// (they may only lie beside one another); one that is written meets those read
// too, and the first that is not allowed ends the search.  Ranges that are read
// never meet, so a tensor that a call lists a million times costs no more than others.
inline mr_status_t check_spans(Span* s, int* open, int n) {
    const auto before = [](const Span& a, const Span& b) { return a.lo < b.lo; };
    if (!std::is_sorted(s, s + n, before)) std::sort(s, s + n, before);
    int reads = 0, writes = n;      // open[0, reads) are read, open[writes, n) written
    for (int i = 0; i < n; ++i) {
        const Span& b = s[i];
        const Span* clash = nullptr;
        const auto ended = [&](const Span& a) {
            if (a.hi <= b.lo) return true;
            if (!allowed(a, b)) clash = &a;
            return false;
        };
        int keep = n;
        for (int j = n - 1; j >= writes && !clash; --j)
            if (!ended(s[open[j]])) open[--keep] = open[j];
        writes = keep;
        if (b.written) {
            keep = 0;
            for (int j = 0; j < reads && !clash; ++j)
                if (!ended(s[open[j]])) open[keep++] = open[j];
            reads = keep;
        }
        if (clash)
            return report_error(MR_ERR_ALIAS, "%s[%d] overlaps %s[%d] in a form that is not an allowed in-place one",
                                clash->name, std::max(0, clash->rank), b.name, std::max(0, b.rank));
        if (b.written) open[--writes] = i;
        else open[reads++] = i;
    }
    return MR_OK;
}
template <int kMost>
mr_status_t check_spans(Spans<kMost>& v) {
    return check_spans(v.s, v.open, v.n);
}

inline bool misaligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

}  // namespace mr
