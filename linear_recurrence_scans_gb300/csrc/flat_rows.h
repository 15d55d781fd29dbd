// Copies of the rows of a dense array in whole 16-byte pieces, `wide` values each.
// A row's pieces are those that hold one of its values, but for the array's last
// piece where that is not whole: nothing beyond the array is read.  (A narrow row
// may end in that piece without being the last one.)
#pragma once

#include <cstdint>

namespace mg {

// Values [flat_copy_begin, flat_copy_end) of the array; empty where end <= begin.
constexpr int64_t flat_copy_begin(int64_t row, int64_t D, int wide) { return row * D / wide * wide; }
constexpr int64_t flat_copy_end(int64_t row, int64_t D, int64_t M, int wide)
{
    const int64_t end = ((row + 1) * D + wide - 1) / wide * wide, whole = M * D / wide * wide;
    return end < whole ? end : whole;
}

}  // namespace mg
