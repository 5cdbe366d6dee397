// schedule.h -- how an expert's rows are dealt to row tiles: plain arithmetic,
// the same on the host and in the kernels.
//
// An expert may own any number of rows below 2^31, so the sums that round up
// are unsigned: n + tiles - 1 passes 2^31 from 2.13e9 rows on (128-row tiles),
// and n + bm - 1 within a tile of the end.
#pragma once

#include <stdint.h>

#include "host_device.h"

namespace moe {

// Row tiles of at most bm rows that n rows take; none for n <= 0.
MOE_HOST_DEVICE int row_tiles_of(int n, int bm) {
    return n > 0 ? static_cast<int>((static_cast<uint32_t>(n) + (bm - 1)) / bm) : 0;
}

// Rows of every one of n's tiles but the last: the even share, rounded up to a
// multiple of gran.  With tiles = row_tiles_of(n, bm) and gran a divisor of bm
// it is at most bm, so the last tile keeps at least one row.
MOE_HOST_DEVICE int rows_per_tile(int n, int tiles, int gran) {
    const uint32_t share = (static_cast<uint32_t>(n) + (tiles - 1)) / tiles;
    return static_cast<int>((share + (gran - 1)) / gran * gran);
}

}  // namespace moe
