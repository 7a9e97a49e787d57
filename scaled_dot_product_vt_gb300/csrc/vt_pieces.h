// Whether the tensors of a call overlap: by their spans, and element by element where the spans meet (heads of one
// projection beside each other, in any nesting).
#pragma once

#include <cstdint>
#include <cstring>

#include "vt_host.h"

#pragma GCC visibility push(hidden)
namespace vt {

// One tensor (or vector) of a call, for the overlap checks.
struct Piece {
    Span span;
    const void *p;
    const int64_t *st;  // nullptr: contiguous
    bool out;
    int side;           // 1: Q's, 2: K's, 3: V's, 0: none of them
    int64_t n[3], D;    // (with st) extents
};
struct Pieces {
    Piece at[20];
    int n = 0;
    void add(const Piece &x) { at[n++] = x; }
};

// Two pieces that are one tensor: reading and writing it in place is allowed.
inline bool same_tensor(const Piece &a, const Piece &b) {
    return a.p == b.p && a.st && b.st && std::memcmp(a.st, b.st, 3 * sizeof(int64_t)) == 0;
}

// A tensor as rows of D elements at every combination of its indices, the largest stride first (indices with one value
// are left out).
struct Grid {
    int64_t n[3], st[3], D;
    int dims = 0;
    explicit Grid(const Piece &x) : D(x.D) {
        for (int i = 0; i < 3; ++i) {
            if (x.n[i] <= 1) continue;
            int at = dims++;
            for (; at > 0 && st[at - 1] < x.st[i]; --at) n[at] = n[at - 1], st[at] = st[at - 1];
            n[at] = x.n[i];
            st[at] = x.st[i];
        }
    }
    // elements from the first to the last one, over the indices from `from` on
    int64_t reach(int from) const {
        int64_t r = D;
        for (int i = from; i < dims; ++i) r += (n[i] - 1) * st[i];
        return r;
    }
};

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }

// Whether an element of a's indices from i on meets one of b's from j on, whose first element lies `delta` elements behind
// a's.  Indices are taken off, the largest stride first and two of one stride together, for those values alone whose
// remainders reach each other: one or two where tensors are parts of one allocation.  Past `steps` of them it says yes.
inline bool meet(const Grid &a, int i, const Grid &b, int j, int64_t delta, int *steps) {
    if (delta >= a.reach(i) || delta + b.reach(j) <= 0) return false;
    if (i == a.dims && j == b.dims) return true;
    const int64_t sa = i < a.dims ? a.st[i] : 0, sb = j < b.dims ? b.st[j] : 0, s = sa > sb ? sa : sb;
    const int i1 = i + (sa == s), j1 = j + (sb == s);
    // a's index minus b's: delta - k s < a's remainder and > minus b's
    int64_t lo = floor_div(delta - a.reach(i1), s) + 1, hi = -floor_div(-(delta + b.reach(j1)), s) - 1;
    const int64_t least = sb == s ? 1 - b.n[j] : 0, most = sa == s ? a.n[i] - 1 : 0;
    if (lo < least) lo = least;
    if (hi > most) hi = most;
    for (int64_t k = lo; k <= hi; ++k)
        if (--*steps < 0 || meet(a, i1, b, j1, delta - k * s, steps)) return true;
    return false;
}

// Two tensors whose spans overlap and whose elements do not: heads beside each other in one projection (Q, K and V side
// by side, in any nesting and width), rows of K and V beside each other in one cache.
inline bool beside(const Piece &x, const Piece &y, int elt) {
    if (!x.st || !y.st) return false;
    const intptr_t bytes = reinterpret_cast<intptr_t>(y.p) - reinterpret_cast<intptr_t>(x.p);
    int steps = 1000;
    return !meet(Grid(x), 0, Grid(y), 0, bytes / elt, &steps);  // (both start on 16 bytes)
}

}  // namespace vt
#pragma GCC visibility pop
