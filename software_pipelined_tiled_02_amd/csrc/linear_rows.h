// linear_rows.h -- whether two matrices in memory have a byte in common.  Host
// code without HIP or torch (tests/host/check_linear_rows.cpp checks it against
// every byte).
#ifndef PIPEGEMM_LINEAR_ROWS_H
#define PIPEGEMM_LINEAR_ROWS_H

#include <stdint.h>

namespace pg {

// `count` rows of `width` bytes, `step` bytes (width or more, where there are two)
// from one to the next.
struct ByteRows { int64_t at, count, width, step; };

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); }       // b > 0

// Rows of one step: by the columns that they take, in one division (the common case:
// columns beside one another).  Others: row by row of the matrix with fewer rows, those
// that lie in the other's range, two divisions each.
inline bool rows_meet(ByteRows x, ByteRows y) {
    if (x.count <= 0 || y.count <= 0 || x.width <= 0 || y.width <= 0) return false;
    if (x.count == 1) x.step = x.width;
    if (y.count == 1) y.step = y.width;
    const int64_t x_end = x.at + (x.count - 1) * x.step + x.width, y_end = y.at + (y.count - 1) * y.step + y.width;
    if (x_end <= y.at || y_end <= x.at) return false;
    if (x.step == y.step) {
        const int64_t d = y.at - x.at - floor_div(y.at - x.at, x.step) * x.step;
        return d < x.width || d + y.width > x.step;
    }
    if (x.count > y.count) {
        const ByteRows z = x;
        x = y;
        y = z;
    }
    const int64_t lo = x.at, hi = y.at + (y.count - 1) * y.step + y.width;
    // x's rows i with an end past y's start and a start before y's end
    int64_t i = floor_div(y.at - lo - x.width, x.step) + 1, last = floor_div(hi - 1 - lo, x.step);
    i = i < 0 ? 0 : i;
    last = last >= x.count ? x.count - 1 : last;
    for (; i <= last; ++i) {
        const int64_t from = x.at + i * x.step - y.at;       // y's rows j: j step + width > from, j step < from + x.width
        int64_t j = floor_div(from - y.width, y.step) + 1;
        j = j < 0 ? 0 : j;
        if (j < y.count && j * y.step < from + x.width) return true;
    }
    return false;
}

}  // namespace pg

#endif
