// How the products of product_tiles.h are cut into workgroups.  Plain arithmetic on sizes,
// with no HIP, so that it is tested on the host.
#pragma once

#include <stdint.h>

namespace mx {

// Tiles of TN columns.
inline int64_t real_columns(int64_t N, int TN) { return (N + TN - 1) / TN; }

// Column tiles per row tile in the launch: from 8 on padded to a multiple of 8 where there
// are several row tiles.  Workgroup b runs on XCD b % 8, so a column tile's workgroups then
// run on one XCD and share its weight rows in one L2.  Fewer than 8 stay as they are: padded,
// every XCD but theirs would get nothing but empty tiles (4096 rows of 16 columns, K = 2880,
// 11.4 -> 4.5 us in MXFP4 and 17.6 -> 5.9 in MXFP8; 8192 rows of 100 columns in 128 x 128
// tiles 33.3 -> 15.6 and 38.9 -> 19.6), and so few weight rows fit every L2.
inline int64_t column_tiles(int64_t M, int64_t N, int TN) {
  const int64_t n = real_columns(N, TN);
  return M > 32 && n >= 8 ? (n + 7) / 8 * 8 : n;
}

}  // namespace mx
