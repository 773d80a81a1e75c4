// Whether two matrices in memory share bytes (host).
#pragma once

#include <stdint.h>

namespace df2 {

struct RowSpan {
    uintptr_t at;
    int64_t row, ld;  // bytes of a row, and from one to the next (ld >= row)
};

// Of N >= 1 rows each.  Rows that are equally far apart, such as two halves of one wide matrix,
// are compared row by row; others by all that lies between their ends.
inline bool rows_share_bytes(const RowSpan& a, const RowSpan& b, int64_t N) {
    const uintptr_t a_end = a.at + uintptr_t(N - 1) * a.ld + a.row, b_end = b.at + uintptr_t(N - 1) * b.ld + b.row;
    if (a.at >= b_end || b.at >= a_end) return false;
    if (a.ld != b.ld || N == 1) return true;
    // b's row j begins d bytes into a's row j + q
    const bool before = b.at < a.at;
    const uintptr_t off = before ? a.at - b.at : b.at - a.at, ld = uintptr_t(a.ld);
    int64_t q = int64_t(off / ld), d = int64_t(off % ld);
    if (before) {
        q = d ? -q - 1 : -q;
        d = d ? a.ld - d : 0;
    }
    const bool with_own = d < a.row && q < N && q > -N, with_next = a.ld - d < b.row && q + 1 < N && q + 1 > -N;
    return with_own || with_next;
}

}  // namespace df2
