// The gated feed-forward block on MX operands for gfx950: both projections,
// the activation and the product in one kernel, and the backward pass that
// recomputes the projections (formulas in gate_device.h).
//
// The kernels here take any shape, element types, scale layout and alignment
// (product_tiles.h); large MXFP4 and MXFP8 / MXFP6 problems go to the 256-row
// pipelines (launch_gated).  Waves that split the K range add their partial tiles
// through LDS in a fixed order.
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

// 128 K-elements of a row: the operand words of two 64-deep steps and the four
// scale bytes, shifted so that byte 0 and byte 2 are this lane's blocks.
template <int F>
struct Piece {
  static constexpr int W = elem_bits<F>();     // words per step
  uint32_t w[2][W];
  int sc;
  __device__ v8i step(int s) const {
    v8i v = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < W; ++k) v[k] = (int)w[s][k];
    return v;
  }
};

// Piece d of the row: K-blocks 4 d .. 4 d + 3, those at nkb and beyond read as
// zero codes at scale 1.  Per step FP4 and FP6 lanes take K-block 2 ks + hi
// whole, FP8 lanes the 16-byte halves [16 hi, +16) of both blocks.  `words`:
// scale rows are 4-byte aligned.
template <int F>
__device__ __forceinline__ void load_piece(Piece<F>& p, const OpRow& r, int d, int nkb, int hi, bool words) {
  const bool full = 4 * d + 4 <= nkb;          // wave-uniform
  if (full && words) {
    p.sc = (int)(*reinterpret_cast<const uint32_t*>(r.scales + 4 * d) >> (8 * hi));
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w |= (4 * d + j < nkb ? (uint32_t)r.scales[4 * d + j] : 127u) << (8 * j);
    p.sc = (int)(w >> (8 * hi));
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int kb = 4 * d + 2 * s;              // the step's first K-block
    uint32_t* const w = p.w[s];
    if constexpr (elem_bits<F>() == 8) {
      uint4 x = make_uint4(0, 0, 0, 0), y = x;
      if (full || kb < nkb) x = *reinterpret_cast<const uint4*>(r.codes + 32 * (int64_t)kb + 16 * hi);
      if (full || kb + 1 < nkb) y = *reinterpret_cast<const uint4*>(r.codes + 32 * (int64_t)kb + 32 + 16 * hi);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
      w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
    } else if constexpr (elem_bits<F>() == 6) {
      uint2 x = make_uint2(0, 0), y = x, z = x;
      if (full || kb + hi < nkb) {
        const uint2* q = reinterpret_cast<const uint2*>(r.codes + 24 * (int64_t)(kb + hi));
        x = q[0], y = q[1], z = q[2];
      }
      w[0] = x.x, w[1] = x.y, w[2] = y.x, w[3] = y.y, w[4] = z.x, w[5] = z.y;
    } else {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (full || kb + hi < nkb) x = *reinterpret_cast<const uint4*>(r.codes + 16 * (int64_t)(kb + hi));
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
  }
}

template <int FA, int FB>
__device__ __forceinline__ v16f mul_piece(const Piece<FA>& a, const Piece<FB>& b, v16f acc) {
  acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a.step(0), b.step(0), acc, mfma_fmt<FA>(), mfma_fmt<FB>(), 0,
                                                         a.sc, 0, b.sc);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a.step(1), b.step(1), acc, mfma_fmt<FA>(), mfma_fmt<FB>(), 2,
                                                          a.sc, 2, b.sc);
}

// One output from its projections.
template <int ACT>
__device__ __forceinline__ void finish(const GatedArgs& a, const GateP& p, int64_t row, int64_t c, float g, float u) {
  if (!a.dH) {
    store_out(a.out, a.out_bf16, row * a.ldo + c, gate_forward<ACT>(p, g, u));
  } else {
    float dg, du;
    gate_backward<ACT>(p, g, u, load_out(a.dH, a.dh_bf16, row * a.lddh + c), dg, du);
    store_out(a.out, a.out_bf16, row * a.ldo + (a.halves ? c : 2 * c), dg);
    store_out(a.out, a.out_bf16, row * a.ldo + (a.halves ? a.N + c : 2 * c + 1), du);
  }
}

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
// Pieces a wave requests before it multiplies the first.  More would cost the
// second workgroup per CU its registers: 64 rows over 32 MXFP8 experts 100 us
// with 2, 145 with 3; MXFP4 53 with 2 or 3, 85 with 4.
constexpr int FD = 2;

template <int FA, int FB, int FW>
__global__ __launch_bounds__(64 * FW) void k_gated_few(GatedArgs a, GateP p, int64_t tiles, int64_t tiles_n,
                                                       int a_words, int b_words) {
  __shared__ float red[FW][32][33];
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t slot = t / tiles_n;
    const int64_t n0 = (t - slot * tiles_n) * 16;
    if (n0 >= a.N) continue;                          // (columns are padded to 8 tiles)
    int ex, rows;
    int64_t row0;
    if (!place_slot<32>(a, slot, ex, row0, rows)) return;   // past the last tile
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l32 = lane & 31, hi = lane >> 5;
    // rows and columns past the end read the last one; their results are dropped
    const int64_t n = n0 + (l32 & 15) < a.N ? n0 + (l32 & 15) : a.N - 1;
    const OpRow ra = op_row(a.A, a.a_2d, row0 + (l32 < rows ? l32 : rows - 1));
    MxOperand B = a.B;
    B.codes += ex * a.stride_codes;
    B.scales += ex * a.stride_scales;
    const OpRow rb = op_row(B, a.b_2d, a.halves ? (int64_t)(l32 >> 4) * a.N + n : 2 * n + (l32 >> 4));
    const int nkb = (int)(a.K / 32), pieces = (nkb + 3) / 4, per = (pieces + FW - 1) / FW;
    const int d0 = w * per, d1 = d0 + per < pieces ? d0 + per : pieces;
    v16f acc = zero16();
    for (int d = d0; d < d1; d += FD) {
      Piece<FA> pa[FD];
      Piece<FB> pb[FD];
#pragma unroll
      for (int i = 0; i < FD; ++i)
        if (d + i < d1) {
          load_piece<FB>(pb[i], rb, d + i, nkb, hi, b_words);
          load_piece<FA>(pa[i], ra, d + i, nkb, hi, a_words);
        }
#pragma unroll
      for (int i = 0; i < FD; ++i)
        if (d + i < d1) acc = mul_piece<FA, FB>(pa[i], pb[i], acc);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) red[w][8 * (r >> 2) + 4 * hi + (r & 3)][l32] = acc[r];
    __syncthreads();
    const int col = threadIdx.x & 15;
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 4 * FW) {
      const int row = r0 + (threadIdx.x >> 4);
      if (row >= rows || n0 + col >= a.N) break;
      float g = red[0][row][col], u = red[0][row][col + 16];
#pragma unroll
      for (int i = 1; i < FW; ++i) {
        g = g + red[i][row][col];
        u = u + red[i][row][col + 16];
      }
      if (p.act == 0) finish<0>(a, p, row0 + row, n0 + col, g, u);
      else if (p.act == 1) finish<1>(a, p, row0 + row, n0 + col, g, u);
      else finish<2>(a, p, row0 + row, n0 + col, g, u);
    }
    __syncthreads();                  // red is free again
  }
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
    const int64_t tiles_n = column_tiles(a.M, a.N, 16), tiles = tiles_n * slot_bound(a, 32);
    if (2 * tiles <= 5 * (int64_t)cu_count())
      hipLaunchKernelGGL((k_gated_few<FA, FB, 8>), dim3(tile_grid(tiles)), dim3(512), 0, st, a, p, tiles, tiles_n,
                         a_words, b_words);
    else
      hipLaunchKernelGGL((k_gated_few<FA, FB, 2>), dim3(tile_grid(tiles)), dim3(128), 0, st, a, p, tiles, tiles_n,
                         a_words, b_words);
  } else {
    const int64_t tiles_n = column_tiles(a.M, a.N, 64), tiles = tiles_n * slot_bound(a, 128);
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
