// Host build of the check for rows that share memory (bit_plane_kv_gb300/csrc/row_ranges.cuh).
#include "row_ranges.cuh"

// x: base, tokens, heads, token step, head step, run
extern "C" int rows_meet(const long long *x, const long long *y) {
    auto set = [](const long long *v) {
        return fathom::RowSet{(uint64_t)v[0], {v[1], v[2]}, {v[3], v[4]}, v[5]};
    };
    return fathom::rows_meet(set(x), set(y));
}
