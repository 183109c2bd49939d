// strided.h -- whether strided tensors with rows of d contiguous elements share memory (host only).
#pragma once

#include <algorithm>
#include <cstdint>

namespace bsattn {

// A [n0, n1, n2, d] tensor of 16-bit elements by its (even) address, its entries and its element strides;
// the stride of a dimension of one entry is never used, all others are positive.
struct Strided {
    const void* base;
    int64_t n[3];
    int64_t stride[3];
    bool same_as(const Strided& o) const {
        for (int i = 0; i < 3; ++i)
            if (n[i] != o.n[i] || (n[i] > 1 && stride[i] != o.stride[i])) return false;
        return base == o.base;
    }
};

namespace strided_detail {

using Wide = __int128;            // 2^31 entries of any 64-bit stride

struct Term {
    Wide stride, lo, hi;          // stride * x, lo <= x <= hi
};

// Whether at + sum of terms can lie in (-d, d).  Terms are sorted, the largest stride first: with the
// nested strides that views of one buffer have, a level leaves two or three values of x to try.  Past
// `budget` of them the answer is yes, to be safe.
inline bool reaches(const Term* t, int terms, Wide at, int d, int& budget) {
    if (terms == 0) return at > -d && at < d;
    Wide low = 0, high = 0;
    for (int i = 1; i < terms; ++i) {
        low += t[i].stride * t[i].lo;
        high += t[i].stride * t[i].hi;
    }
    // stride * x lies in [a, b]
    const Wide a = 1 - d - at - high, b = d - 1 - at - low, s = t[0].stride;
    const Wide from = std::max(t[0].lo, a >= 0 ? (a + s - 1) / s : -((-a) / s));
    const Wide to = std::min(t[0].hi, b >= 0 ? b / s : -((-b + s - 1) / s));
    for (Wide x = from; x <= to; ++x)
        if (--budget < 0 || reaches(t + 1, terms - 1, at + s * x, d, budget)) return true;
    return false;
}

inline void add_term(Term* t, int& terms, Wide stride, Wide lo, Wide hi) {
    for (int i = 0; i < terms; ++i)
        if (t[i].stride == stride) {
            t[i].lo += lo;
            t[i].hi += hi;
            return;
        }
    t[terms++] = {stride, lo, hi};
}

inline bool reaches_sorted(Term* t, int terms, Wide at, int d) {
    std::sort(t, t + terms, [](const Term& x, const Term& y) { return x.stride > y.stride; });
    int budget = 20000;
    return reaches(t, terms, at, d, budget);
}

}  // namespace strided_detail

// Whether an element of a is an element of b.
inline bool overlap(const Strided& a, const Strided& b, int d) {
    using namespace strided_detail;
    Term t[6];
    int terms = 0;
    for (int i = 0; i < 3; ++i) {
        if (a.n[i] > 1) add_term(t, terms, a.stride[i], 0, a.n[i] - 1);
        if (b.n[i] > 1) add_term(t, terms, b.stride[i], 1 - b.n[i], 0);
    }
    const Wide at = (static_cast<Wide>(reinterpret_cast<uintptr_t>(a.base)) - reinterpret_cast<uintptr_t>(b.base)) / 2;
    Wide low = at, high = at;                     // most tensors lie apart as a whole
    for (int i = 0; i < terms; ++i) {
        low += t[i].stride * t[i].lo;
        high += t[i].stride * t[i].hi;
    }
    return high > -d && low < d && reaches_sorted(t, terms, at, d);
}

// Whether two of a's rows share an element.
inline bool overlaps_itself(const Strided& a, int d) {
    using namespace strided_detail;
    // most are nested: each stride at least the extent of all smaller ones
    Term all[3];
    int dims = 0;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] > 1) all[dims++] = {a.stride[i], 0, a.n[i] - 1};
    std::sort(all, all + dims, [](const Term& x, const Term& y) { return x.stride < y.stride; });
    Wide extent = d;
    bool nested = true;
    for (int i = 0; i < dims; ++i) {
        nested = nested && all[i].stride >= extent;
        extent += all[i].stride * all[i].hi;
    }
    if (nested) return false;
    // the difference of two rows: dimension `first` is the first that differs, and taken to be positive
    for (int first = 0; first < 3; ++first) {
        if (a.n[first] <= 1) continue;
        Term t[3];
        int terms = 0;
        t[terms++] = {a.stride[first], 1, a.n[first] - 1};
        for (int i = first + 1; i < 3; ++i)
            if (a.n[i] > 1) add_term(t, terms, a.stride[i], 1 - a.n[i], a.n[i] - 1);
        if (reaches_sorted(t, terms, 0, d)) return true;
    }
    return false;
}

}  // namespace bsattn
