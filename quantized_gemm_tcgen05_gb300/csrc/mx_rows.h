// Row blocks of rows sorted by expert: the integer rules that the 4-bit kernels
// apply to offsets of any value, compiled for host and device, so the host tests
// check the very code the kernels run.
#pragma once
#include "work_sched.h"

namespace qg {

// n plus the blocks of bm rows that rows lo .. hi - 1 make, at most `most`: a
// partition of the rows never has more, and offsets that are none (they may promise
// 2^32 rows an expert) then cost no more time than one that is.
QG_HD int32_t mx_add_blocks(int32_t n, int32_t lo, int32_t hi, int bm, int32_t most) {
    const int64_t m = (int64_t)hi - lo;
    const int64_t sum = n + (m > 0 ? (m + bm - 1) / bm : 0);
    return sum < most ? (int32_t)sum : most;
}

// Where the rows lo .. hi - 1 of an expert end that have scales: its first row lies
// on atom row `tiles` (the atom rows of the experts before it), and there are
// rows / 128 + experts atom rows.  A partition of the rows never reaches that limit.
// An expert that starts before row 0 has none.
QG_HD int64_t mx_span_end(int64_t lo, int64_t hi, int64_t tiles, int64_t rows, int32_t experts) {
    const int64_t room = rows / 128 + experts - tiles;
    if (lo < 0 || room <= 0) return lo;
    return hi - lo < room * 128 ? hi : lo + room * 128;
}

}  // namespace qg
