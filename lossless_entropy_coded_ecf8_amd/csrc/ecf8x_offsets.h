// ecf8x_offsets.h -- where the lanes of a product's tiles read the rows' scales.
// Nothing of the GPU's is needed here: a host compiler takes it too.
#ifndef ECF8X_OFFSETS_H
#define ECF8X_OFFSETS_H

#include <cstdint>

namespace ecf8x {

// A tile's rows of scales are sent for in parts of 8 * each rows, `each` by a wave, one a lane: the row of a lane, and its
// byte offset from the tile's first one, `pitch` bytes a row.  Of the tile's rows `rows` exist; lanes past them take the last
// one, whose scales then reach no result that is stored.  (The range of a buffer is no guard here: it need not count the
// scalar offset, which holds the place inside of a row.)
constexpr int scale_row(int part, int wave, int lane, int each) { return (part * 8 + wave) * each + lane; }

constexpr uint32_t scale_offset(int part, int wave, int lane, int each, int64_t rows, uint32_t pitch)
{
    const int row = scale_row(part, wave, lane, each);
    return (uint32_t)(row < rows ? row : rows - 1) * pitch;
}

}  // namespace ecf8x

#endif
