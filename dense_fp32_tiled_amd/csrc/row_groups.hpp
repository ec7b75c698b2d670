// row_groups.hpp -- the arithmetic of groups of rows (host and device,
// constexpr): which rows a group has, and how many tiles or chunks lie before
// it.
//
// Offsets come from the caller's device memory and need not ascend.  Clamped
// one by one they keep every group inside the matrix, but groups may then
// overlap and have more tiles between them than any division of the rows: up
// to 65535 times all of the rows.  Counts of that size do not fit 32 bits, so
// they are cut at the number of places there are before they are added up.
#pragma once

#include <stdint.h>

namespace dft {

// Group g's rows [lo, hi): offsets outside [0, rows] or not ascending are
// taken as the nearest range inside, so that no access leaves the matrices.
struct RowRange {
    int64_t lo, hi;
    constexpr int64_t tiles(int64_t tile_rows) const { return (hi - lo + tile_rows - 1) / tile_rows; }
};
constexpr RowRange group_rows(const int32_t* offsets, int g, int64_t rows) {
    const int64_t a = offsets[g], b = offsets[g + 1];
    const int64_t lo = a < 0 ? 0 : a > rows ? rows : a;
    const int64_t hi = b < lo ? lo : b > rows ? rows : b;
    return RowRange{lo, hi};
}

// A count of at most `most` (below 2^31).
constexpr int count_at_most(int64_t count, int64_t most) { return (int)(count < most ? count : most); }

}  // namespace dft
