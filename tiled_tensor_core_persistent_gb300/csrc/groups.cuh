// groups.cuh -- reading a device table of row offsets: what the grouped
// block-scaled products and the column quantiser share.
#pragma once

#include <cuda_runtime.h>

namespace tcg {

// Groups g0 .. g0 + 31 of a device table of offsets (lane l has group g0 + l):
// rows [row, row + len) of the group, none past the last group.  Offsets are
// clamped into [0, rows], and one below an earlier one counts as that one
// (`last`: the largest so far, 0 before the first call), so the groups of any
// table lie one after the other, hold at most `rows` rows together and name
// none that does not exist.  For a whole warp.
__device__ __forceinline__ void group_rows(const int* offsets, int groups, int rows, int g0, int lane, int& last, int& row,
                                           int& len) {
    const int g = g0 + lane;
    int r = 0, end = 0;
    if (g < groups) {
        r = min(max(__ldg(offsets + g), 0), rows);
        end = min(max(__ldg(offsets + g + 1), 0), rows);
    }
    r = max(r, last);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, r, d);
        if (lane >= d) r = max(r, o);
    }
    row = r;
    len = g < groups ? max(end - r, 0) : 0;
    last = __shfl_sync(0xffffffffu, r, 31);
}

}  // namespace tcg
