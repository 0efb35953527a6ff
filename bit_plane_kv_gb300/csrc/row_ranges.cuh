// row_ranges.cuh -- whether two sets of strided rows share a byte.  Plain arithmetic, for the
// argument checks and for a host test.
#pragma once

#include <cstdint>

namespace fathom {

// Rows (token, head) of `run` bytes at base + token * step[0] + head * step[1].
struct RowSet {
    uint64_t base;
    int64_t count[2], step[2], run;
};

using wide_int = __int128;   // strides of 2^40 bytes times 2^28 tokens

inline wide_int floor_div(wide_int a, wide_int b) { return a / b - (a % b != 0 && (a < 0) != (b < 0)); }

// Whether runs [0, ra) + i h, i < na, and [d, d + rb) + j h, j < nb, share a byte: some m = j - i
// with -rb < d + m h < ra.
inline bool runs_meet(wide_int d, wide_int ra, wide_int na, wide_int rb, wide_int nb, wide_int h) {
    wide_int lo = -(na - 1), hi = nb - 1;
    if (h == 0) return -rb < d && d < ra;
    const wide_int from = floor_div(-rb - d, h) + 1, to = -floor_div(-(ra - d), h) - 1;
    if (from > lo) lo = from;
    if (to < hi) hi = to;
    return lo <= hi;
}

// False only where no byte is shared.  Exact for sets whose token steps and whose head steps
// are equal (an axis of one entry has any step); others count as meeting where their extents do.
inline bool rows_meet(const RowSet &a, const RowSet &b) {
    const wide_int delta = (wide_int)b.base - (wide_int)a.base;
    auto extent = [](const RowSet &x, int axis) { return (wide_int)(x.count[axis] - 1) * (x.count[axis] > 1 ? x.step[axis] : 0); };
    const wide_int all_a = extent(a, 0) + extent(a, 1) + a.run, all_b = extent(b, 0) + extent(b, 1) + b.run;
    if (delta >= all_a || delta + all_b <= 0) return false;
    auto step = [&](int axis, bool &same) {
        if (a.count[axis] > 1 && b.count[axis] > 1 && a.step[axis] != b.step[axis]) same = false;
        return (wide_int)(a.count[axis] > 1 ? a.step[axis] : b.count[axis] > 1 ? b.step[axis] : 0);
    };
    for (int outer = 0; outer < 2; ++outer) {   // tokens around heads, or heads around tokens
        const int inner = 1 - outer;
        bool same = true;
        const wide_int S = step(outer, same);
        if (!same) continue;
        const wide_int h = step(inner, same);   // same: whether the inner steps are too
        const wide_int span_a = extent(a, inner) + a.run, span_b = extent(b, inner) + b.run;
        wide_int lo = -(wide_int)(a.count[outer] - 1), hi = b.count[outer] - 1;
        if (S) {   // the distances k S at which the inner extents meet
            const wide_int from = floor_div(-span_b - delta, S) + 1, to = -floor_div(-(span_a - delta), S) - 1;
            if (from > lo) lo = from;
            if (to < hi) hi = to;
        } else {
            lo = hi = 0;
        }
        if (hi - lo > 64) continue;
        bool meet = false;
        for (wide_int k = lo; k <= hi && !meet; ++k) {
            const wide_int d = delta + k * S;
            meet = same ? runs_meet(d, a.run, a.count[inner], b.run, b.count[inner], h) : -span_b < d && d < span_a;
        }
        if (!meet) return false;
    }
    return true;
}

}  // namespace fathom
