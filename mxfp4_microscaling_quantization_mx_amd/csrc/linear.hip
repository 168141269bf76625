// The linear layer on MX operands for gfx950, its bias, activation and residual in the
// product's epilogue:
//   Y = act(A B^T + bias) + residual,
// and the backward pass through the activation, the product recomputed:
//   dP = dY * act'(A B^T + bias)
// (activations in gate_device.h), dense or with a weight and bias per expert.
//
// The kernels here take any shape, element types, scale layout and alignment
// (product_tiles.h); large MXFP4 and MXFP8 / MXFP6 problems go to the 256-row
// pipelines (the rule is in launch_rule.h).
//  * k_linear_rows16: 16 rows by 16 columns per workgroup of 8, 4 or 2 waves, which
//    split K.  For few rows, where reading the weight once with as many loads in flight as
//    possible is all that counts.
//  * k_linear_tile: 128 rows by 128 columns per workgroup of 8 waves, operands
//    staged through a ring in LDS.  1037 x 1451 x 2912 MXFP8 backward 21.3 us: 108
//    workgroups of 23 stages, 0.6 us each, on 256 CUs.
#include "product_tiles.h"

namespace mx {

namespace {

// ---------------------------------------------------------------- 16 x 16 tiles
// V_MFMA_SCALE_F32_16X16X128_F8F6F4: lane l holds row (or column) l % 16 and, g = l / 16,
// K-block g of a 128-deep piece (FP8: bytes [16 g, +16) of its first and of its second
// half) with that block's scale.  Straight loads of that would take 16 bytes from 16 rows
// for every 16 neighbouring lanes, one address at a time.  Instead the four lanes 4 r ..
// 4 r + 3 load the four blocks of row r, 64 to 128 neighbouring bytes, and the words change
// lanes in registers (ds_bpermute): 16 rows of 11264 x 4096 MXFP4 11.3 -> 8.4 us, 32 rows
// 17.7 -> 12.1.  A wave has BD pieces of 16 columns in flight, 256 to 512 neighbouring bytes
// of each; 32 columns by half as many bytes (32X32X64) used half of the CUs for one row.
//
// One row of N = K = 2880 4.4 us (MXFP8 5.9; 5.4 and 7.7 with 32 x 32 tiles): the launch, one
// trip to memory along K and one for the epilogue.  1 x 65536 x 2880 (101 MB) 20.5 (5 TB/s),
// 64 rows over 32 experts, 22 of them with rows, 27-29 (97 MB; MXFP8 42-48, 188 MB): HBM
// bandwidth, and two trips to memory before the first weights arrive.
constexpr int BD = 4;                     // pieces of a batch: 16 blocks, 256 to 512 bytes of a row
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t scale_words4 __attribute__((ext_vector_type(4)));
typedef scale_words4 loose_scales __attribute__((aligned(1)));

// Pieces [d, d1) of a row, BD of them at most; blocks at nkb and beyond as zero codes at
// scale 1.
template <int F>
struct Batch {
  static constexpr int W = elem_bits<F>();
  uint32_t w[BD][W];
  scale_words4 sc;                        // byte g of word i: block g of piece i

  __device__ __forceinline__ void load(const OpRow& r, int d, int d1, int nkb, int g) {
    const bool full = 4 * (d + BD) <= nkb;       // wave-uniform
    if (full) {
      sc = *reinterpret_cast<const loose_scales*>(r.scales + 4 * d);
    } else {
#pragma unroll
      for (int i = 0; i < BD; ++i) {
        const int kb = 4 * (d + i) + g;
        sc[i] = (kb < nkb ? (uint32_t)r.scales[kb] : 127u) << (8 * g);
      }
    }
#pragma unroll
    for (int i = 0; i < BD; ++i) {
      if (d + i >= d1) break;
      const int kb = 4 * (d + i);
      uint32_t* const q = w[i];
      if constexpr (elem_bits<F>() == 8) {
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        const uint8_t* const c = r.codes + 32 * (int64_t)kb + 16 * g;
        if (full || kb + (g >> 1) < nkb) x = *reinterpret_cast<const uint4*>(c);
        if (full || kb + 2 + (g >> 1) < nkb) y = *reinterpret_cast<const uint4*>(c + 64);
        q[0] = x.x, q[1] = x.y, q[2] = x.z, q[3] = x.w;
        q[4] = y.x, q[5] = y.y, q[6] = y.z, q[7] = y.w;
      } else if constexpr (elem_bits<F>() == 6) {
        uint2 x = make_uint2(0, 0), y = x, z = x;
        if (full || kb + g < nkb) {
          const uint2* const c = reinterpret_cast<const uint2*>(r.codes + 24 * (int64_t)(kb + g));
          x = c[0], y = c[1], z = c[2];
        }
        q[0] = x.x, q[1] = x.y, q[2] = y.x, q[3] = y.y, q[4] = z.x, q[5] = z.y;
      } else {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (full || kb + g < nkb) x = *reinterpret_cast<const uint4*>(r.codes + 16 * (int64_t)(kb + g));
        q[0] = x.x, q[1] = x.y, q[2] = x.z, q[3] = x.w;
      }
    }
  }
  // Byte i: the scale of the block that this lane multiplies of piece i.
  __device__ __forceinline__ int scales(int g, int from) const {
    const uint32_t pick = 0x0400u + 0x0101u * g;
    const uint32_t lo = __builtin_amdgcn_perm(sc[1], sc[0], pick), hi = __builtin_amdgcn_perm(sc[3], sc[2], pick);
    return __builtin_amdgcn_ds_bpermute(from, (int)__builtin_amdgcn_perm(hi, lo, 0x05040100u));
  }
  template <int I>
  __device__ __forceinline__ v8i piece(int from) const {
    v8i v = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < W; ++k) v[k] = __builtin_amdgcn_ds_bpermute(from, (int)w[I][k]);
    return v;
  }
};

template <int FA, int FB, int I>
__device__ __forceinline__ v4f mul_at(const Batch<FA>& a, const Batch<FB>& b, int sa, int sb, int from, v4f acc) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.template piece<I>(from), b.template piece<I>(from), acc,
                                                          mfma_fmt<FA>(), mfma_fmt<FB>(), I, sa, I, sb);
}

template <int FA, int FB, int FW>
__global__ __launch_bounds__(64 * FW) void k_linear_rows16(LinearArgs a, GateP p, int64_t tiles, int64_t tiles_n) {
  __shared__ float red[FW][16][17];
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t slot = t / tiles_n, n0 = (t - slot * tiles_n) * 16;
    if (n0 >= a.N) continue;                          // (columns are padded to 8 tiles)
    int ex, rows;
    int64_t row0;
    if (!place_slot<16>(a, slot, ex, row0, rows)) return;   // past the last tile
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // where this lane loads, where it multiplies and the lane that loads that
    const int rl = lane >> 2, gl = lane & 3, l16 = lane & 15, g = lane >> 4, from = 4 * (4 * l16 + g);
    // rows and columns past the end read the last one; their results are dropped
    const OpRow ra = op_row(a.A, a.a_2d, row0 + (rl < rows ? rl : rows - 1));
    MxOperand B = a.B;
    B.codes += ex * a.stride_codes;
    B.scales += ex * a.stride_scales;
    const OpRow rb = op_row(B, a.b_2d, n0 + rl < a.N ? n0 + rl : a.N - 1);
    const int nkb = (int)(a.K / 32), pieces = (nkb + 3) / 4, per = (pieces + FW - 1) / FW;
    const int d0 = w * per, d1 = d0 + per < pieces ? d0 + per : pieces;
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
    // this thread's bias, and its first pass's residual: float32 ones come while the products
    // run, bf16 ones (shifted where they are loaded) are waited for here
    const int col = threadIdx.x & 15, first = threadIdx.x >> 4;
    float bias = 0.0f, r_first = 0.0f;
    if (n0 + col < a.N) {
      bias = linear_bias(a, ex, n0 + col);
      if (a.dH && first < rows) r_first = load_out(a.dH, a.dh_bf16, (row0 + first) * a.lddh + n0 + col);
    }
    for (int d = d0; d < d1; d += BD) {
      Batch<FA> ba;
      Batch<FB> bb;
      bb.load(rb, d, d1, nkb, gl);
      ba.load(ra, d, d1, nkb, gl);
      const int sa = ba.scales(gl, from), sb = bb.scales(gl, from);
      acc = mul_at<FA, FB, 0>(ba, bb, sa, sb, from, acc);
      if (d + 1 < d1) acc = mul_at<FA, FB, 1>(ba, bb, sa, sb, from, acc);
      if (d + 2 < d1) acc = mul_at<FA, FB, 2>(ba, bb, sa, sb, from, acc);
      if (d + 3 < d1) acc = mul_at<FA, FB, 3>(ba, bb, sa, sb, from, acc);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) red[w][4 * g + r][l16] = acc[r];
    __syncthreads();
#pragma unroll 1
    for (int row = first; row < rows && n0 + col < a.N; row += 4 * FW) {
      float x = red[0][row][col];
#pragma unroll
      for (int i = 1; i < FW; ++i) x = x + red[i][row][col];
      const float r = row == first || !a.dH ? r_first : load_out(a.dH, a.dh_bf16, (row0 + row) * a.lddh + n0 + col);
      store_out(a.out, a.out_bf16, (row0 + row) * a.ldo + n0 + col, linear_out(a, p, x + bias, r));
    }
    __syncthreads();                  // red is free again
  }
}

template <int FA, int FB>
__global__ __launch_bounds__(512) void k_linear_tile(LinearArgs a, GateP p, int64_t tiles, int64_t tiles_n, int a_words,
                                                     int b_words) {
  row_tiles<true, FA, FB>(a, p, tiles, tiles_n, a_words, b_words);
}

template <int FA, int FB, int FW>
void launch_rows16(const LinearArgs& a, const GateP& p, int64_t tiles, int64_t tiles_n, hipStream_t st) {
  hipLaunchKernelGGL((k_linear_rows16<FA, FB, FW>), dim3(tile_grid(tiles)), dim3(64 * FW), 0, st, a, p, tiles, tiles_n);
}

template <int FA, int FB>
hipError_t launch_direct(const LinearArgs& a, bool few, hipStream_t st) {
  const GateP p = gate_params(a.act, a.alpha, a.limit, a.up_shift);
  if (few || !row_tiles_fit<true>(a)) {
    const int64_t tiles_n = column_tiles(a.M, a.N, 16), tiles = tiles_n * slot_bound(a, 16);
    const int waves = rows16_waves(a.M, a.N, a.offsets ? a.E : 0, cu_count());
    if (waves == 8) launch_rows16<FA, FB, 8>(a, p, tiles, tiles_n, st);
    else if (waves == 4) launch_rows16<FA, FB, 4>(a, p, tiles, tiles_n, st);
    else launch_rows16<FA, FB, 2>(a, p, tiles, tiles_n, st);
  } else {
    const Words w = scale_words(a);
    const int64_t tiles_n = column_tiles(a.M, a.N, 128), tiles = tiles_n * slot_bound(a, 128);
    hipLaunchKernelGGL((k_linear_tile<FA, FB>), dim3(tile_grid(tiles)), dim3(512), 0, st, a, p, tiles, tiles_n, w.a,
                       w.b);
  }
  return hipGetLastError();
}

template <int FA>
hipError_t launch_direct_b(const LinearArgs& a, bool few, hipStream_t st) {
  switch (a.b_elem) {
    case 1: return launch_direct<FA, 1>(a, few, st);
    case 2: return launch_direct<FA, 2>(a, few, st);
    case 3: return launch_direct<FA, 3>(a, few, st);
    case 4: return launch_direct<FA, 4>(a, few, st);
    default: return launch_direct<FA, 0>(a, few, st);
  }
}

}  // namespace

// (the rule and what it was measured by: launch_rule.h)
hipError_t launch_linear(const LinearArgs& a, hipStream_t st) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  const LinearKernel kernel = linear_kernel(a.M, a.N, a.offsets ? a.E : 0, a.a_elem == 0 && a.b_elem == 0,
                                            a.b_elem == 1 || a.b_elem == 2, cu_count());
  const bool few = kernel == LinearKernel::ROWS16;
  if (kernel == LinearKernel::PIPELINE) {
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
