// The linear layer on MX operands for gfx950, its bias, activation and residual in the
// product's epilogue:
//   Y = act(A B^T + bias) + residual,
// and the backward pass through the activation, the product recomputed:
//   dP = dY * act'(A B^T + bias)
// (activations in gate_device.h), dense or with a weight and bias per expert.
//
// The kernels here take any shape, element types, scale layout and alignment
// (product_tiles.h); large MXFP4 and MXFP8 / MXFP6 problems go to the 256-row
// pipelines (launch_linear).
//  * k_linear_few: 32 rows by 32 columns per workgroup of 8 or 2 waves, which split K.
//    For few rows, where reading the weight once with as many loads in flight as
//    possible is all that counts.
//    One row of N = K = 2880 5.2 us (9.0 with the call): the launch, two trips along K and
//    one to the output for 4.2 MB.
//  * k_linear_tile: 128 rows by 128 columns per workgroup of 8 waves, operands
//    staged through a ring in LDS.  1037 x 1451 x 2912 MXFP8 backward 21.4 us: 108
//    workgroups of 23 stages, 0.6 us each, on 256 CUs.
#include "product_tiles.h"

namespace mx {

namespace {

template <int FA, int FB, int FW>
__global__ __launch_bounds__(64 * FW) void k_linear_few(GatedArgs a, GateP p, int64_t tiles, int64_t tiles_n,
                                                        int a_words, int b_words) {
  few_rows<true, FA, FB, FW>(a, p, tiles, tiles_n, a_words, b_words);
}

template <int FA, int FB>
__global__ __launch_bounds__(512) void k_linear_tile(GatedArgs a, GateP p, int64_t tiles, int64_t tiles_n, int a_words,
                                                     int b_words) {
  row_tiles<true, FA, FB>(a, p, tiles, tiles_n, a_words, b_words);
}

template <int FA, int FB>
hipError_t launch_direct(const GatedArgs& a, bool few, hipStream_t st) {
  const GateP p = gate_params(a.act, a.alpha, a.limit, a.up_shift);
  const Words w = scale_words(a);
  if (few || !row_tiles_fit<true>(a)) {
    const int64_t tiles_n = column_tiles(a, 32), tiles = tiles_n * slot_bound(a, 32);
    if (2 * tiles <= 5 * (int64_t)cu_count())
      hipLaunchKernelGGL((k_linear_few<FA, FB, 8>), dim3(tile_grid(tiles)), dim3(512), 0, st, a, p, tiles, tiles_n, w.a,
                         w.b);
    else
      hipLaunchKernelGGL((k_linear_few<FA, FB, 2>), dim3(tile_grid(tiles)), dim3(128), 0, st, a, p, tiles, tiles_n, w.a,
                         w.b);
  } else {
    const int64_t tiles_n = column_tiles(a, 128), tiles = tiles_n * slot_bound(a, 128);
    hipLaunchKernelGGL((k_linear_tile<FA, FB>), dim3(tile_grid(tiles)), dim3(512), 0, st, a, p, tiles, tiles_n, w.a,
                       w.b);
  }
  return hipGetLastError();
}

template <int FA>
hipError_t launch_direct_b(const GatedArgs& a, bool few, hipStream_t st) {
  switch (a.b_elem) {
    case 1: return launch_direct<FA, 1>(a, few, st);
    case 2: return launch_direct<FA, 2>(a, few, st);
    case 3: return launch_direct<FA, 3>(a, few, st);
    case 4: return launch_direct<FA, 4>(a, few, st);
    default: return launch_direct<FA, 0>(a, few, st);
  }
}

}  // namespace

// Which kernel (us as k_linear_few / k_linear_tile / pipeline, N = K = 2880 unless said,
// bias and residual, graph replays; MXFP4, then MXFP8):
//  * k_linear_few while its workgroups are at most 2 per CU: 1 row 5.1 / 13.2 / 25 (7.2 /
//    17.7 / 51), 128 rows 11.7 / 13.4 (17.6 / 19.6), 128 of 4096 x 4096 15.5 / 19.8 (23.3 /
//    25.9); 192 rows 16.9 / 13.9 (24.1 / 19.2), 64 of 11264 x 4096 25.9 / 18.2 (37.6 /
//    23.9).  Grouped over 32 experts 16 rows 16.0 / 16.7 (27.1 / 22.7), 64 rows 41.3 / 41.5
//    (65 / 57), 256 rows 59 / 50 (90 / 69).
//  * k_linear_tile while one workgroup per CU does in MXFP4, two with wider elements: 1280
//    rows 19.5 / 28.0, 1400 33.1 / 28.3; 2048 rows (39.7 / 55.2), 3000 (58.5 / 56.0).  Grouped
//    in MXFP4 up to 16 rows per expert (32 experts: 512 rows 53.4 / 57.5, 768 63.8 / 58.3; 128
//    of 1024 x 2048: 1024 rows 50 / 46, 8192 73 / 64) or 5 workgroups per 4 CUs (8 of 4096 x
//    4096: 256 rows 21.3 / 30.7, 1024 39 / 32), up to 128 with wider elements (32 experts:
//    2048 rows 94 / 114, 4096 119 / 118, 8192 180 / 167; 8 of 4096 x 4096: 1024 69 / 85,
//    4096 159 / 151).  Also everything that the pipelines do not take.
//  * the 256-row pipelines beyond.
hipError_t launch_linear(const GatedArgs& a, hipStream_t st) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  const int64_t cus = cu_count();
  const int64_t few_wgs = (a.N + 31) / 32 * slot_bound(a, 32), tile_wgs = column_tiles(a, 128) * slot_bound(a, 128);
  const bool f4 = a.a_elem == 0 && a.b_elem == 0;
  const bool few = few_wgs <= 2 * cus;
  const bool tile = a.offsets ? a.M <= (f4 ? 16 : 128) * (int64_t)a.E || (f4 && 4 * tile_wgs <= 5 * cus)
                              : tile_wgs <= (f4 ? 1 : 2) * cus;
  if (!few && !tile) {
    if (linear256_layout_ok(a)) return launch_linear256(a, st);
    if (linear_f8_layout_ok(a)) return launch_linear_f8(a, st);
  }
  switch (a.a_elem) {
    case 1: return launch_direct_b<1>(a, few, st);
    case 2: return launch_direct_b<2>(a, few, st);
    case 3: return launch_direct_b<3>(a, few, st);
    case 4: return launch_direct_b<4>(a, few, st);
    default: return launch_direct_b<0>(a, few, st);
  }
}

}  // namespace mx
