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
//  * k_linear_tile: 128 rows by 128 columns per workgroup of 8 waves, operands
//    staged through a ring in LDS.
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

// Which kernel: as for the gated block (launch_gated), whose tiles hold as many weight
// rows for half as many columns.
hipError_t launch_linear(const GatedArgs& a, hipStream_t st) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  const int64_t cus = cu_count();
  const int64_t few_wgs = (a.N + 31) / 32 * slot_bound(a, 32), tile_wgs = (a.N + 127) / 128 * slot_bound(a, 128);
  const bool f4 = a.a_elem == 0 && a.b_elem == 0;
  const bool few = a.offsets ? a.M <= 8 * (int64_t)a.E || few_wgs <= 6 * cus : 2 * few_wgs <= (f4 ? 6 : 5) * cus;
  if (!few && (a.offsets || tile_wgs > (f4 ? 1 : 2) * cus)) {
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
