// k2t_rows.h -- host-side checks of tensors [rows, heads, dim] that the calls
// of a model that reads a graph share.
#pragma once

#include <cstdint>

namespace k2t {

// Rows of 16-byte pieces, with pitches that a tensor map holds (40 bits of bytes).
inline bool rows_aligned(const void *p, int64_t row, int64_t head)
{
    return !((uintptr_t)p & 15u) && !(row & 7) && !(head & 7) && row >= 0 && head >= 0 && row < (1ll << 38) && head < (1ll << 38);
}

// Whether two rows of an output [rows, heads, d] share values: rows i apart and heads j apart the other way, |i row - j head| < d.
inline bool rows_overlap(int64_t row, int64_t head, uint64_t rows, uint64_t heads, uint32_t d)
{
    using Wide = unsigned __int128;
    if ((rows > 1 && row < d) || (heads > 1 && head < d)) return true;
    if (rows < 2 || heads < 2) return false;
    if (row >= (Wide)(heads - 1) * head + d || head >= (Wide)(rows - 1) * row + d) return false;     // one inside the other
    for (uint64_t j = 1; j < heads; ++j) {
        const Wide at = (Wide)j * head, i = at / row, left = at - i * row;
        if ((i < rows && left < d) || (i + 1 < rows && row - left < d)) return true;
    }
    return false;
}

}  // namespace k2t
