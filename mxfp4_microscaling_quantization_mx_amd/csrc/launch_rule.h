// How the products of product_tiles.h are cut into workgroups, and which of its kernels the
// linear layer takes.  Plain arithmetic on sizes, with no HIP, so that it is tested on the
// host.
#pragma once

#include <stdint.h>

namespace mx {

// Column tiles per row tile in the launch: from 8 on padded to a multiple of 8 where there
// are several row tiles.  Workgroup b runs on XCD b % 8, so a column tile's workgroups then
// run on one XCD and share its weight rows in one L2.  Fewer than 8 stay as they are: padded,
// every XCD but theirs would get nothing but empty tiles (4096 rows of 16 columns, K = 2880,
// 11.4 -> 4.5 us in MXFP4 and 17.6 -> 5.9 in MXFP8; 8192 rows of 100 columns in 128 x 128
// tiles 33.3 -> 15.6 and 38.9 -> 19.6), and so few weight rows fit every L2.
inline int64_t column_tiles(int64_t M, int64_t N, int TN) {
  const int64_t n = (N + TN - 1) / TN;
  return M > 32 && n >= 8 ? (n + 7) / 8 * 8 : n;
}

// Row tiles of TM rows; of E experts (0: not grouped) the most that a launch must offer:
// every expert with rows adds at most one partial tile.
inline int64_t row_tiles_bound(int64_t M, int64_t E, int TM) {
  return E == 0 ? (M + TM - 1) / TM : M / TM + (E < M ? E : M);
}

enum class LinearKernel { ROWS16, TILE, PIPELINE };

// Which kernel runs a linear layer (E experts, 0: not grouped; f4: both operands MXFP4; wide:
// an 8-bit weight).  Workgroups are counted as launched: an eighth of the padded number is
// what the busiest XCD gets (1400 rows of 2880 columns: 253 of 264 are real, and one CU of
// seven XCDs has two).  us as k_linear_rows16 / k_linear_tile / pipeline, N = K = 2880 unless
// said, bias and residual, graph replays; MXFP4, then MXFP8:
//  * k_linear_rows16 for one row tile, and while its workgroups are at most 8 per CU: 1 row of
//    65536 20.5 / 32.2 (39 / 51), 32 rows 38 / 28 (78 / 48); 160 rows 11.3 / 14.3 (16.8 / 18.6),
//    192 12.8 / 14.4 (18.9 / 18.9), 256 16.1 / 14.9 (22.8 / 19.0); 64 of 11264 x 4096 18.7 /
//    17.2 (32.7 / 27.4); 512 of 1024 x 4096 13.2 / 17.8 (20.7 / 23.6).  Narrow, K = 2880: 16384
//    rows of 16 columns 9.0 / 14.9 / 25 (13.2 / 19.8 / 49), 4096 of 100 13.1 / 14.4 / 24 (20.5 /
//    18.8 / 48), 8192 of 100 22.6 / 15.6 / 24 (35.5 / 19.6 / 49).  Grouped also up to 16
//    rows per expert, 12 of an 8-bit weight, whose bytes count for more where experts have
//    two row tiles: over 32 experts 64 rows 27.2 / 42.9 (41.5 / 61.3), 256 rows 40.7 / 54
//    (63 / 78), 512 rows 47 / 49.5 (77 / 69), 1024 rows 63.5 / 54.8; over 128 of 1024 x 2048
//    2048 rows 46.9 / 57.6 (75.8 / 79); over 8 of 4096 x 4096 128 rows 25.0 / 22.1 (41 / 39).
//  * k_linear_tile while one workgroup per CU does in MXFP4, two with wider elements: 1280
//    rows 19.5 / 28.0 (tile, pipeline), 1400 33.1 / 28.3; 2048 rows (39.7 / 55.2),
//    3000 (58.5 / 56.0); 8192 rows of 400 columns 21.2 / 28.9 (24.8 / 51.8), 16384 of 400 39.4 /
//    31 (47 / 53), of 640 51.9 / 32 (66.7 / 55.8).  Grouped in MXFP4 up to 5 workgroups per
//    4 CUs if every expert had a partial tile (8 of 4096 x 4096: 256 rows 21.3 / 30.7, 1024 39 /
//    32; 32 experts: 768 rows 63.8 / 58.3), and below 8 column tiles, where many row tiles make
//    that number and most are whole, one per CU if half of the experts had (8 of 400 columns:
//    2048 rows 17.4 / 24.3, 8192 33.9 / 26.1; 32 of 128: 16384 rows 19.3 / 25.3, of 200 34.5 /
//    26.1).  With wider elements up to 128 rows per expert or 2 workgroups per CU (32
//    experts: 2048 rows 94 / 114, 4096 119 / 118, 8192 180 / 167; 8 of 4096 x 4096: 1024 69 / 85,
//    4096 159 / 151; 8 of 128 columns: 16384 rows 22.4 / 48; 32 of 400: 8192 rows 43.5 / 49.1,
//    16384 65.9 / 49.8).  Also everything that the pipelines do not take.
//  * the 256-row pipelines beyond.
inline LinearKernel linear_kernel(int64_t M, int64_t N, int64_t E, bool f4, bool wide, int64_t cus) {
  const int64_t few = column_tiles(M, N, 16) * row_tiles_bound(M, E, 16);
  if (few <= 8 * cus || (E ? M <= (wide ? 12 : 16) * E : M <= 16)) return LinearKernel::ROWS16;
  const int64_t n = column_tiles(M, N, 128), tile = n * row_tiles_bound(M, E, 128);
  if (!E) return tile <= (f4 ? 1 : 2) * cus ? LinearKernel::TILE : LinearKernel::PIPELINE;
  const bool fits = f4 ? 4 * tile <= 5 * cus && (n >= 8 || n * (2 * (M / 128) + E) <= 2 * cus) : M <= 128 * E || tile <= 2 * cus;
  return fits ? LinearKernel::TILE : LinearKernel::PIPELINE;
}

// Waves of k_linear_rows16's workgroups, which split K: us of 8, 4 and 2, 1 x 2880 x 2880 4.4,
// 4.8, 6.0; 64 rows 8.9, 6.7, 8.3; 128 rows 12.8, 10.6, 9.5; 64 rows over 32 experts 46, 29.4,
// 27.2; 8192 rows of 16 columns 5.8, 6.2, 7.4, 16384 10.8, 9.0, 9.8.
inline int rows16_waves(int64_t M, int64_t N, int64_t E, int64_t cus) {
  const int64_t tiles = column_tiles(M, N, 16) * row_tiles_bound(M, E, 16);
  return tiles <= 2 * cus ? 8 : tiles <= 5 * cus ? 4 : 2;
}

}  // namespace mx
