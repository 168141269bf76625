// Bias gradients for gfx950: the sums of a matrix's columns over all its rows, or
// over the rows of each expert.
//
// Bound by HBM bandwidth: every element is read once.  The rows are cut into tiles
// of BG_ROWS (a tile never spans two experts), a workgroup sums one tile's columns
// in float32, its waves each every 16th row and then the waves in order through
// LDS, and a second launch adds an expert's tiles in order: no atomics, the same
// bits on every run.  Few rows are summed straight to the result in one launch.
#include "group_device.h"
#include "row_device.h"
#include "mx_launch.h"

namespace mx {

namespace {

constexpr int BG_WAVES = 16;
constexpr int BG_ROWS = 256;
constexpr int BG_UNROLL = 4;              // rows a wave has requested at once
constexpr int64_t BG_DIRECT = 512;        // rows up to which one launch does

template <bool BF16>
constexpr int slab_cols() { return 64 * RowPiece<BF16>::VEC; }

// Sums of rows [row0, row0 + rows) over this workgroup's columns from c0, in wave 0
// after the call: element i of lane l is column c0 + VEC l + i.
template <bool BF16>
__device__ __forceinline__ void tile_sum(const BiasGradArgs& a, int64_t row0, int64_t rows, int64_t c0,
                                         float (*red)[64 * 8 + 4], RowPiece<BF16>& acc) {
  using P = RowPiece<BF16>;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = c0 + lane * P::VEC;
  const int n = (int)(c >= a.N ? 0 : a.N - c < P::VEC ? a.N - c : P::VEC);
  acc.zero();
  const char* const p = static_cast<const char*>(a.dp) + (row0 * a.ld + c) * P::ES;
  const int64_t ldb = a.ld * P::ES;
  if (n > 0) {
    int64_t r = w;
    for (; r + (BG_UNROLL - 1) * BG_WAVES < rows; r += BG_UNROLL * BG_WAVES) {
      typename P::words q[BG_UNROLL];
#pragma unroll
      for (int i = 0; i < BG_UNROLL; ++i) q[i] = P::load(p + (r + i * BG_WAVES) * ldb, n);
#pragma unroll
      for (int i = 0; i < BG_UNROLL; ++i) {
        P x;
        x.unpack(q[i]);
#pragma unroll
        for (int k = 0; k < P::VEC; ++k) acc.v[k] = acc.v[k] + x.v[k];
      }
    }
    for (; r < rows; r += BG_WAVES) {
      P x;
      x.unpack(P::load(p + r * ldb, n));
#pragma unroll
      for (int k = 0; k < P::VEC; ++k) acc.v[k] = acc.v[k] + x.v[k];
    }
  }
  // halves of the waves onto the other half, four times
#pragma unroll
  for (int h = BG_WAVES / 2; h > 0; h >>= 1) {
    __syncthreads();
    if (w >= h && w < 2 * h) {
#pragma unroll
      for (int k = 0; k < P::VEC; ++k) red[w - h][k * 64 + lane] = acc.v[k];
    }
    __syncthreads();
    if (w < h) {
#pragma unroll
      for (int k = 0; k < P::VEC; ++k) acc.v[k] = acc.v[k] + red[w][k * 64 + lane];
    }
  }
}

__device__ __forceinline__ void put_sum(const BiasGradArgs& a, int64_t i, float v) {
  if (a.out_bf16) static_cast<uint16_t*>(a.out)[i] = (uint16_t)f32_to_bf16_rne(v);
  else static_cast<float*>(a.out)[i] = v;
}

// blockIdx.x: column slab, blockIdx.y: expert; all of its rows.
template <bool BF16>
__global__ __launch_bounds__(64 * BG_WAVES) void k_bias_direct(BiasGradArgs a) {
  __shared__ float red[BG_WAVES / 2][64 * 8 + 4];
  const int64_t c0 = (int64_t)blockIdx.x * slab_cols<BF16>();
  for (int e = blockIdx.y; e < a.E; e += gridDim.y) {
    int64_t lo = 0, hi = a.M;
    if (a.offsets) expert_rows(a.offsets, e, a.M, lo, hi);
    RowPiece<BF16> acc;
    tile_sum<BF16>(a, lo, hi - lo, c0, red, acc);
    if (threadIdx.x < 64) {
#pragma unroll
      for (int k = 0; k < RowPiece<BF16>::VEC; ++k) {
        const int64_t c = c0 + threadIdx.x * RowPiece<BF16>::VEC + k;
        if (c < a.N) put_sum(a, e * a.N + c, acc.v[k]);
      }
    }
  }
}

// blockIdx.x: row tile and column slab; ws[tile][N].
template <bool BF16>
__global__ __launch_bounds__(64 * BG_WAVES) void k_bias_part(BiasGradArgs a, uint32_t slabs) {
  __shared__ float red[BG_WAVES / 2][64 * 8 + 4];
  const int64_t slot = blockIdx.x / slabs;
  const int64_t c0 = (int64_t)(blockIdx.x - (uint32_t)slot * slabs) * slab_cols<BF16>();
  int ex = 0, rows;
  int64_t row0 = slot * BG_ROWS;
  if (a.offsets) {
    if (!find_slot<BG_ROWS>(a.offsets, a.E, a.M, slot, ex, row0, rows)) return;   // past the last tile
  } else {
    rows = (int)(a.M - row0 < BG_ROWS ? a.M - row0 : BG_ROWS);
  }
  RowPiece<BF16> acc;
  tile_sum<BF16>(a, row0, rows, c0, red, acc);
  if (threadIdx.x < 64) {
#pragma unroll
    for (int k = 0; k < RowPiece<BF16>::VEC; ++k) {
      const int64_t c = c0 + threadIdx.x * RowPiece<BF16>::VEC + k;
      if (c < a.N) a.ws[slot * a.N + c] = acc.v[k];
    }
  }
}

// blockIdx.x: 64 columns, blockIdx.y: expert.  Wave w adds the tiles w, w + 4, ...
// and the four sums are added in order.
__global__ __launch_bounds__(256) void k_bias_sum(BiasGradArgs a) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  for (int e = blockIdx.y; e < a.E; e += gridDim.y) {
    int64_t lo = 0, hi = a.M, s0 = 0;
    if (a.offsets) {
      expert_rows(a.offsets, e, a.M, lo, hi);
      s0 = slots_before<BG_ROWS>(a.offsets, e, a.M);
    }
    const int64_t tiles = (hi - lo + BG_ROWS - 1) / BG_ROWS;
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

template <bool BF16>
hipError_t launch_bias_grad_t(const BiasGradArgs& a, hipStream_t st) {
  const int64_t slabs = (a.N + slab_cols<BF16>() - 1) / slab_cols<BF16>();
  const unsigned ey = (unsigned)(a.E < 65535 ? a.E : 65535);
  if (a.M <= BG_DIRECT) {
    hipLaunchKernelGGL((k_bias_direct<BF16>), dim3((unsigned)slabs, ey), dim3(64 * BG_WAVES), 0, st, a);
    return hipGetLastError();
  }
  const int64_t tiles = tile_bound(a.M, a.E, a.offsets != nullptr);
  hipLaunchKernelGGL((k_bias_part<BF16>), dim3((unsigned)(tiles * slabs)), dim3(64 * BG_WAVES), 0, st, a,
                     (uint32_t)slabs);
  hipLaunchKernelGGL(k_bias_sum, dim3((unsigned)((a.N + 63) / 64), ey), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

size_t bias_grad_workspace(int64_t M, int64_t N, int32_t E, bool grouped) {
  return M <= BG_DIRECT ? 0 : (size_t)tile_bound(M, E, grouped) * (size_t)N * sizeof(float);
}
bool bias_grad_fits(int64_t M, int64_t N, int32_t E, bool grouped) {
  return tile_bound(M, E, grouped) * ((N + 255) / 256) < (1ll << 31);
}

hipError_t launch_bias_grad(const BiasGradArgs& a, hipStream_t st) {
  return a.bf16 ? launch_bias_grad_t<true>(a, st) : launch_bias_grad_t<false>(a, st);
}

}  // namespace mx
