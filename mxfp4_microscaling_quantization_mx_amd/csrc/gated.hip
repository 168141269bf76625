// The gated feed-forward block on MX operands for gfx950: both projections,
// the activation and the product in one kernel, and the backward pass that
// recomputes the projections (formulas in gate_device.h).
//
// The kernels here take any shape, element types, scale layout and alignment
// (product_tiles.h); large MXFP4 and MXFP8 / MXFP6 problems go to the 256-row
// pipelines (launch_gated).
//  * k_gated_few: 32 rows by 16 hidden columns per workgroup of 8 or 2 waves,
//    which split K; the B tile is the 32 weight rows of the columns' gates
//    (first 16) and ups (last 16).  For few rows, where reading the weight
//    once with as many loads in flight as possible is all that counts.
//  * k_gated_tile: 128 rows by 64 hidden columns per workgroup of 8 waves,
//    operands staged through a ring in LDS; a wave's two B tiles are its
//    columns' gates and ups.
#include "product_tiles.h"

namespace mx {

namespace {

// k_gated_few reads every weight byte once per 32 rows straight into MFMA
// operand registers; its FW waves split K.  8 waves up to 2.5 workgroups per CU,
// so that 2880 columns are 180 workgroups with loads in flight on every CU; 2
// beyond, where a wave's longer walk along K has its loads in flight for more
// of a workgroup's life and 20 waves fit a CU (16 as two workgroups of 8).  us
// with 8, 4, 2 and 1 waves: 128 x 2880 x 2880 MXFP4 15.6, 13.1, 13.6, 16.1 (90
// rows 12.5, 12.9, 13.2, 15.3); 64 rows over 32 experts, 22 of them with rows,
// 53, 48, 43, 45 (MXFP8 100, 96, 95, 104), and 52-56 with the weights out of
// the caches (59-62 with 8): 3.6 TB/s.  One row of N = K = 2880 takes 4.6 us on
// the GPU (8.8 MB of weights that earlier runs left in the caches) and 7.8 with
// the call.
template <int FA, int FB, int FW>
__global__ __launch_bounds__(64 * FW) void k_gated_few(GatedArgs a, GateP p, int64_t tiles, int64_t tiles_n,
                                                       int a_words, int b_words) {
  few_rows<false, FA, FB, FW>(a, p, tiles, tiles_n, a_words, b_words);
}

// 512 x 2880 x 2880: MXFP4 17.8 us, MXFP8 23.4, of which 7.5 are the launch, the
// first loads and the epilogue, and the rest 0.41 and 0.67 us per stage: 10 and
// 12 TB/s out of the XCDs' L2s, which a larger tile would lower and leave CUs
// idle for.  Staged through registers with two LDS buffers: 18.9 and 28.2.
// RING 3 or 5 (with a remainder to take per stage) costs MXFP4 1 us, MXFP8
// none; 8 slots MXFP4 1 us.
template <int FA, int FB>
__global__ __launch_bounds__(512) void k_gated_tile(GatedArgs a, GateP p, int64_t tiles, int64_t tiles_n, int a_words,
                                                    int b_words) {
  row_tiles<false, FA, FB>(a, p, tiles, tiles_n, a_words, b_words);
}

template <int FA, int FB>
hipError_t launch_direct(const GatedArgs& a, bool few, hipStream_t st) {
  const GateP p = gate_params(a.act, a.alpha, a.limit, a.up_shift);
  const int a_words = scale_words(a).a, b_words = scale_words(a).b;
  if (few || !row_tiles_fit<false>(a)) {
    const int64_t tiles_n = column_tiles(a, 16), tiles = tiles_n * slot_bound(a, 32);
    if (2 * tiles <= 5 * (int64_t)cu_count())
      hipLaunchKernelGGL((k_gated_few<FA, FB, 8>), dim3(tile_grid(tiles)), dim3(512), 0, st, a, p, tiles, tiles_n,
                         a_words, b_words);
    else
      hipLaunchKernelGGL((k_gated_few<FA, FB, 2>), dim3(tile_grid(tiles)), dim3(128), 0, st, a, p, tiles, tiles_n,
                         a_words, b_words);
  } else {
    const int64_t tiles_n = column_tiles(a, 64), tiles = tiles_n * slot_bound(a, 128);
    hipLaunchKernelGGL((k_gated_tile<FA, FB>), dim3(tile_grid(tiles)), dim3(512), 0, st, a, p, tiles, tiles_n, a_words,
                       b_words);
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

// Which kernel (us, N = K = 2880 unless said; MXFP4, then MXFP8):
//  * k_gated_few while its workgroups are at most 3 per CU in MXFP4, 2.5 with
//    wider elements: 128 rows 13.6 against k_gated_tile's 16.2 (23.7 / 21.8),
//    192 rows 21 / 16.5 (38 / 22), 256 rows of 1440 x 2912 16.1 / 16.1 (24.1 /
//    21.7), 192 rows 13.4 / 16.0 (20.3 / 21.4).  Grouped, whose weights are read
//    from HBM, up to 8 rows per expert (32 experts, 64 rows 43 against the
//    pipeline's 68, 256 rows 70 / 78, 512 rows about 90 / 83; MXFP8 95 / 140, 136
//    / 147) or 6 workgroups per CU (512 x 1024: 512 rows 11 / 15, 1024 rows 15 /
//    15).  Wide weights (K = 4096, out of the caches) leave it: with 32 rows of
//    14336 columns it takes 29 against k_gated_tile's 21, with 32 of 28672 50
//    against the pipeline's 35 (MXFP8 82 / 65); with a single row 20 / 22 and 35 /
//    36 (MXFP8 33 / 31, 11008 columns 23 / 27).
//  * k_gated_tile while one workgroup per CU does in MXFP4, 16-18 against the
//    21-24 of a pipeline that is not full and 32 with two; while two do with
//    wider elements, 22-24 with one, 43 with two against the pipeline's 47-49
//    (MXFP6 41-43 / 40-45).  Also everything that the pipelines do not take.
//  * the 256-row pipelines beyond, and for groups (2048 rows over 32 experts 89
//    against k_gated_tile's 125; MXFP8 169 / 182).
hipError_t launch_gated(const GatedArgs& a, hipStream_t st) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  const int64_t cus = cu_count();
  const int64_t few_wgs = (a.N + 15) / 16 * slot_bound(a, 32), tile_wgs = (a.N + 63) / 64 * slot_bound(a, 128);
  const bool f4 = a.a_elem == 0 && a.b_elem == 0;
  const bool few = a.offsets ? a.M <= 8 * (int64_t)a.E || few_wgs <= 6 * cus : 2 * few_wgs <= (f4 ? 6 : 5) * cus;
  if (!few && (a.offsets || tile_wgs > (f4 ? 1 : 2) * cus)) {
    if (gated256_layout_ok(a)) return launch_gated256(a, st);
    if (gated_f8_layout_ok(a)) return launch_gated_f8(a, st);
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
