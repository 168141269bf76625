// Bias gradients for gfx950: the sums of a matrix's columns over all its rows, or
// over the rows of each expert.
//
// Bound by HBM bandwidth: every element is read once.  The rows are cut into tiles
// of BG_ROWS (a tile never spans two experts), a workgroup sums one tile's columns
// in float32, its waves each every 16th row (or every 64th for each quarter of a
// wave) and then those sums in order through LDS, and a second launch adds an
// expert's tiles in order: no atomics, the same bits on every run.  Up to BG_DIRECT
// rows are summed straight to the result in one launch.  A wave takes 64 pieces of a
// row, or 16 pieces of four rows where 64 would leave CUs idle: 1037 x 1451 bf16 6.9 us
// for 13.8, 512 x 2880 3.8 for 7.5.  65536 x 2880 bf16 over 32 experts 69 us (5.5 TB/s)
// and 5 for the second launch, 16384 x 2880 20.0 for both.
#include "group_device.h"
#include "row_device.h"
#include "mx_launch.h"

namespace mx {

namespace {

constexpr int BG_WAVES = 16;
constexpr int BG_ROWS = 256;
constexpr int BG_UNROLL = 4;              // rows a lane has requested at once
constexpr int64_t BG_DIRECT = 1024;       // rows up to which one launch does

// Columns of a workgroup whose waves take LPR pieces of a row.
template <bool BF16, int LPR>
constexpr int slab_cols() { return LPR * RowPiece<BF16>::VEC; }

// Sums of rows [row0, row0 + rows) over this workgroup's columns from c0: thread t <
// slab_cols returns that of column c0 + t.
template <bool BF16, int LPR>
__device__ __forceinline__ float tile_sum(const BiasGradArgs& a, int64_t row0, int64_t rows, int64_t c0, float* red) {
  using P = RowPiece<BF16>;
  constexpr int COLS = slab_cols<BF16, LPR>(), STEP = BG_WAVES * 64 / LPR;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane & (LPR - 1);
  const int64_t c = c0 + g * P::VEC;
  const int n = (int)(c >= a.N ? 0 : a.N - c < P::VEC ? a.N - c : P::VEC);
  P acc;
  acc.zero();
  const char* const p = static_cast<const char*>(a.dp) + (row0 * a.ld + c) * P::ES;
  const int64_t ldb = a.ld * P::ES;
  if (n > 0) {
    int64_t r = w * (64 / LPR) + lane / LPR;
    for (; r + (BG_UNROLL - 1) * STEP < rows; r += BG_UNROLL * STEP) {
      typename P::words q[BG_UNROLL];
#pragma unroll
      for (int i = 0; i < BG_UNROLL; ++i) q[i] = P::load(p + (r + i * STEP) * ldb, n);
#pragma unroll
      for (int i = 0; i < BG_UNROLL; ++i) {
        P x;
        x.unpack(q[i]);
#pragma unroll
        for (int k = 0; k < P::VEC; ++k) acc.v[k] = acc.v[k] + x.v[k];
      }
    }
    for (; r < rows; r += STEP) {
      P x;
      x.unpack(P::load(p + r * ldb, n));
#pragma unroll
      for (int k = 0; k < P::VEC; ++k) acc.v[k] = acc.v[k] + x.v[k];
    }
  }
  if constexpr (LPR == 16) {              // the wave's four rows: lanes 16 and 32 apart
#pragma unroll
    for (int k = 0; k < P::VEC; ++k) {
      uint32_t u = __float_as_uint(acc.v[k]);
      const auto x = __builtin_amdgcn_permlane16_swap(u, u, false, false);
      u = __float_as_uint(__uint_as_float(x[0]) + __uint_as_float(x[1]));
      const auto y = __builtin_amdgcn_permlane32_swap(u, u, false, false);
      acc.v[k] = __uint_as_float(y[0]) + __uint_as_float(y[1]);
    }
  }
  __syncthreads();                        // red may still be read by the previous sum
  if (lane < LPR) {
#pragma unroll
    for (int k = 0; k < P::VEC; ++k) red[w * COLS + k * LPR + g] = acc.v[k];
  }
  __syncthreads();
  // column t is element t % VEC of lane t / VEC
  const int t = threadIdx.x;
  float s = 0.0f;
  if (t < COLS) {
    const float* const q = red + (t % P::VEC) * LPR + t / P::VEC;
    s = q[0];
#pragma unroll
    for (int i = 1; i < BG_WAVES; ++i) s = s + q[i * COLS];
  }
  return s;
}

__device__ __forceinline__ void put_sum(const BiasGradArgs& a, int64_t i, float v) {
  if (a.out_bf16) static_cast<uint16_t*>(a.out)[i] = (uint16_t)f32_to_bf16_rne(v);
  else static_cast<float*>(a.out)[i] = v;
}

// blockIdx.x: column slab, blockIdx.y: expert; all of its rows.
template <bool BF16, int LPR>
__global__ __launch_bounds__(64 * BG_WAVES) void k_bias_direct(BiasGradArgs a) {
  constexpr int COLS = slab_cols<BF16, LPR>();
  __shared__ float red[BG_WAVES * COLS];
  const int64_t c0 = (int64_t)blockIdx.x * COLS, c = c0 + threadIdx.x;
  for (int e = blockIdx.y; e < a.E; e += gridDim.y) {
    int64_t lo = 0, hi = a.M;
    if (a.offsets) expert_rows(a.offsets, e, a.M, lo, hi);
    const float s = tile_sum<BF16, LPR>(a, lo, hi - lo, c0, red);
    if (threadIdx.x < COLS && c < a.N) put_sum(a, e * a.N + c, s);
  }
}

// blockIdx.x: row tile and column slab; ws[tile][N].
template <bool BF16, int LPR>
__global__ __launch_bounds__(64 * BG_WAVES) void k_bias_part(BiasGradArgs a, uint32_t slabs) {
  constexpr int COLS = slab_cols<BF16, LPR>();
  __shared__ float red[BG_WAVES * COLS];
  const int64_t slot = blockIdx.x / slabs;
  const int64_t c0 = (int64_t)(blockIdx.x - (uint32_t)slot * slabs) * COLS, c = c0 + threadIdx.x;
  int ex = 0, rows;
  int64_t row0 = slot * BG_ROWS;
  if (a.offsets) {
    if (!find_slot<BG_ROWS>(a.offsets, a.E, a.M, slot, ex, row0, rows)) return;   // past the last tile
  } else {
    rows = (int)(a.M - row0 < BG_ROWS ? a.M - row0 : BG_ROWS);
  }
  const float s = tile_sum<BF16, LPR>(a, row0, rows, c0, red);
  if (threadIdx.x < COLS && c < a.N) a.ws[slot * a.N + c] = s;
}

// blockIdx.x: 64 columns, blockIdx.y: expert.  Wave w adds the tiles w, w + 4, ...
// and the four sums are added in order.  (Offsets that decrease may name more tiles
// than the `bound` that ws holds; those past it are left out.)
__global__ __launch_bounds__(256) void k_bias_sum(BiasGradArgs a, int64_t bound) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  for (int e = blockIdx.y; e < a.E; e += gridDim.y) {
    int64_t lo = 0, hi = a.M, s0 = 0;
    if (a.offsets) {
      expert_rows(a.offsets, e, a.M, lo, hi);
      s0 = slots_before<BG_ROWS>(a.offsets, e, a.M);
    }
    int64_t tiles = (hi - lo + BG_ROWS - 1) / BG_ROWS;
    if (tiles > bound - s0) tiles = bound - s0;
    float s = 0.0f;
    if (c < a.N)
#pragma unroll 8
      for (int64_t i = w; i < tiles; i += 4) s = s + a.ws[(s0 + i) * a.N + c];
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < a.N) put_sum(a, e * a.N + c, ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane]);
    __syncthreads();
  }
}

int64_t tile_bound(int64_t M, int32_t E, bool grouped) {
  return grouped ? M / BG_ROWS + (E < M ? E : M) : (M + BG_ROWS - 1) / BG_ROWS;
}

template <bool BF16, int LPR>
hipError_t launch_bias_grad_t(const BiasGradArgs& a, hipStream_t st) {
  const int64_t slabs = (a.N + slab_cols<BF16, LPR>() - 1) / slab_cols<BF16, LPR>();
  const unsigned ey = (unsigned)(a.E < 65535 ? a.E : 65535);
  if (a.M <= BG_DIRECT) {
    hipLaunchKernelGGL((k_bias_direct<BF16, LPR>), dim3((unsigned)slabs, ey), dim3(64 * BG_WAVES), 0, st, a);
    return hipGetLastError();
  }
  const int64_t tiles = tile_bound(a.M, a.E, a.offsets != nullptr);
  hipLaunchKernelGGL((k_bias_part<BF16, LPR>), dim3((unsigned)(tiles * slabs)), dim3(64 * BG_WAVES), 0, st, a,
                     (uint32_t)slabs);
  hipLaunchKernelGGL(k_bias_sum, dim3((unsigned)((a.N + 63) / 64), ey), dim3(256), 0, st, a, tiles);
  return hipGetLastError();
}

// 64 pieces of a row per wave where that makes two workgroups per CU, else 16 pieces of
// four rows (see above).
template <bool BF16>
hipError_t launch_bias_grad_w(const BiasGradArgs& a, hipStream_t st) {
  const int64_t slabs = (a.N + slab_cols<BF16, 64>() - 1) / slab_cols<BF16, 64>();
  const int64_t wgs = slabs * (a.M <= BG_DIRECT ? a.E : tile_bound(a.M, a.E, a.offsets != nullptr));
  return wgs >= 2 * cu_count() ? launch_bias_grad_t<BF16, 64>(a, st) : launch_bias_grad_t<BF16, 16>(a, st);
}

}  // namespace

size_t bias_grad_workspace(int64_t M, int64_t N, int32_t E, bool grouped) {
  return M <= BG_DIRECT ? 0 : (size_t)tile_bound(M, E, grouped) * (size_t)N * sizeof(float);
}
// (a launch has fewer than 2^32 threads along an axis, a workgroup 1024 and at least
// 256 columns where there are many)
bool bias_grad_fits(int64_t M, int64_t N, int32_t E, bool grouped) {
  const int64_t tiles = tile_bound(M, E, grouped);
  return (tiles < 1 ? 1 : tiles) * ((N + 255) / 256) < (1ll << 22);
}

hipError_t launch_bias_grad(const BiasGradArgs& a, hipStream_t st) {
  return a.bf16 ? launch_bias_grad_w<true>(a, st) : launch_bias_grad_w<false>(a, st);
}

}  // namespace mx
