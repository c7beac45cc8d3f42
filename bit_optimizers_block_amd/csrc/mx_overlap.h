// mx_overlap.h -- whether two matrices in memory share a byte.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace bitopt {

// `rows` rows of `width` bytes, `stride` bytes apart (stride >= width where there are several).
struct ByteRows {
    const void* p;
    int64_t rows, width, stride;
};

// Exact also where the rows of one lie between those of the other: halves of a wider buffer do
// not meet.  128 bits, since no bound on the distance of rows is checked elsewhere.
inline bool rows_meet(const ByteRows& x, const ByteRows& y) {
    typedef __int128 wide;
    if (!x.p || !y.p || x.rows <= 0 || y.rows <= 0 || x.width <= 0 || y.width <= 0) return false;
    const ByteRows &a = x.rows <= y.rows ? x : y, &b = x.rows <= y.rows ? y : x;
    const wide pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const wide sb = b.rows > 1 ? b.stride : b.width, sa = a.rows > 1 ? a.stride : sb;
    if (pa >= pb + (b.rows - 1) * sb + b.width || pb >= pa + (a.rows - 1) * sa + a.width) return false;
    auto floor_div = [](wide n, wide d) { return n / d - (n % d < 0 ? 1 : 0); };
    // Row i of a meets row j of b when -a.width < d < b.width, d = pa - pb + i sa - j sb.  With one
    // stride only t = i - j counts, from `lo` to `hi`; with two, every row of a is a matrix of one row.
    auto some = [&](wide d0, int64_t rows) {
        const wide lo = std::max<wide>(floor_div(-a.width - d0, sb) + 1, 1 - b.rows);
        const wide hi = std::min<wide>(-floor_div(d0 - b.width, sb) - 1, rows - 1);
        return lo <= hi;
    };
    if (sa == sb) return some(pa - pb, a.rows);
    for (int64_t i = 0; i < a.rows; ++i)
        if (some(pa - pb + i * sa, 1)) return true;
    return false;
}

}  // namespace bitopt
