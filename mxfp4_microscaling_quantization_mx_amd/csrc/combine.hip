// Rows to their places sorted by expert and back for gfx950 (dest[t, j]: the
// sorted row of token t's j-th choice; outside [0, rows) the choice was dropped):
//   dispatch          xs[dest[t, j]] = x[t]
//   combine           out[t] = sum_j w[t, j] y[dest[t, j]] + residual[t]
//   combine backward  dy[dest[t, j]] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[dest[t, j]]>
// Sums in float32 in the order of j (dw: in an order fixed by the width), rounded
// once.  All three are driven from the tokens, so that each token's row is read
// once and no result needs an atomic.
//
// Bound by HBM bandwidth (a device copy 5.05 TB/s): 16384 x 2880 bf16, 4 choices, combine
// 90 us without and 105-107 with a residual (478 MB read, 94 written, 5.3 TB/s), backward
// 160-162 (5.3), dispatch 79 (6.0).  In wide rows a lane has the whole 16-byte pieces of its
// choices, four at a time, in flight at once, which is enough beside the other waves of a
// CU.  Two things do not overlap:
//  * a row's last piece where it is not whole: its elements are loaded one at a time, in bf16
//    each waited for before the next, up to 7 per choice.  4099 x 1111 bf16 16.0 us, at a
//    stride of 1112 too, and 10.3 with 1112 columns; backward 31 and 17.6; 16384 x 2879 110
//    and 91 with 2880.  In float32 (up to 3 elements) 17.7 with either, backward 41 and 34.
//  * rows of at most 32 pieces, laid side by side: each lane reads its own entries of dest
//    and waits for one before it requests that choice's row.  The backward pass gives every
//    token a workgroup, whatever its width, and reads dest and weights first: 8192 x 32, 64
//    or 128 columns 9 us.
#include "row_device.h"
#include "mx_launch.h"

namespace mx {

namespace {

constexpr int CK = 4;                     // choices taken at a time

// Row `d` of a choice, or row 0 with ok false (which every caller may read: there
// is at least one row).
__device__ __forceinline__ int64_t choice_row(int32_t d, int64_t rows, bool& ok) {
  ok = d >= 0 && d < rows;
  return ok ? d : 0;
}

// This lane's row and piece: a wave takes 64 pieces of one row (WIDE), or rows of
// up to 2^shift pieces side by side.
struct Place {
  int64_t row;
  int64_t c;                              // first element of the piece
};
template <bool WIDE, int VEC>
__device__ __forceinline__ Place piece_place(uint32_t parts, int shift) {
  const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const uint32_t lane = threadIdx.x & 63;
  if constexpr (WIDE) {
    const uint32_t row = wave / parts;
    return {(int64_t)row, (int64_t)((wave - row * parts) * 64 + lane) * VEC};
  }
  return {((int64_t)wave << (6 - shift)) + (lane >> shift), (int64_t)(lane & ((1u << shift) - 1)) * VEC};
}

template <bool BF16, bool WIDE>
__global__ __launch_bounds__(256) void k_combine(CombineArgs a, uint32_t parts, int shift) {
  using P = RowPiece<BF16>;
  const Place p = piece_place<WIDE, P::VEC>(parts, shift);
  if (p.row >= a.T || p.c >= a.C) return;
  const int n = (int)(a.C - p.c < P::VEC ? a.C - p.c : P::VEC);
  const int32_t* const dest = a.dest + p.row * a.top;
  const float* const w = a.weights ? a.weights + p.row * a.top : nullptr;
  const char* const y = static_cast<const char*>(a.y) + p.c * P::ES;
  typename P::words r = {0u, 0u, 0u, 0u};
  if (a.residual) r = P::load(static_cast<const char*>(a.residual) + (p.row * a.ldr + p.c) * P::ES, n);
  P acc;
  acc.zero();
  for (int j0 = 0; j0 < a.top; j0 += CK) {
    typename P::words q[CK];
    float f[CK];
    bool ok[CK];
#pragma unroll
    for (int j = 0; j < CK; ++j) {
      const bool in = j0 + j < a.top;
      const int64_t d = choice_row(in ? dest[j0 + j] : -1, a.rows, ok[j]);
      f[j] = in && w ? w[j0 + j] : 1.0f;
      q[j] = P::load(y + d * a.ldy * P::ES, n);
    }
#pragma unroll
    for (int j = 0; j < CK; ++j) {
      P x;
      x.unpack(q[j]);
#pragma unroll
      for (int i = 0; i < P::VEC; ++i) acc.v[i] = ok[j] ? __builtin_fmaf(f[j], x.v[i], acc.v[i]) : acc.v[i];
    }
  }
  if (a.residual) {
    P x;
    x.unpack(r);
#pragma unroll
    for (int i = 0; i < P::VEC; ++i) acc.v[i] = acc.v[i] + x.v[i];
  }
  P::store(static_cast<char*>(a.out) + (p.row * a.ldo + p.c) * P::ES, acc.pack(), n);
}

template <bool BF16, bool WIDE>
__global__ __launch_bounds__(256) void k_dispatch(CombineArgs a, uint32_t parts, int shift) {
  using P = RowPiece<BF16>;
  const Place p = piece_place<WIDE, P::VEC>(parts, shift);
  if (p.row >= a.T || p.c >= a.C) return;
  const int n = (int)(a.C - p.c < P::VEC ? a.C - p.c : P::VEC);
  const int32_t* const dest = a.dest + p.row * a.top;
  const typename P::words x = P::load(static_cast<const char*>(a.dout) + (p.row * a.lddo + p.c) * P::ES, n);
  char* const xs = static_cast<char*>(a.dy) + p.c * P::ES;
  for (int j = 0; j < a.top; ++j) {
    bool ok;
    const int64_t d = choice_row(dest[j], a.rows, ok);
    if (ok) P::store(xs + d * a.lddy * P::ES, x, n);
  }
}

// One token per workgroup of NW waves: every lane takes every (64 NW)-th piece of
// the row, writes the choices' gradients and keeps its part of their dot products.
template <bool BF16, int NW>
__global__ __launch_bounds__(64 * NW) void k_combine_backward(CombineArgs a) {
  using P = RowPiece<BF16>;
  __shared__ float red[2][NW][CK];        // (by turns, so that one barrier a chunk of choices does)
  const int64_t t = blockIdx.x;
  const char* const dout = static_cast<const char*>(a.dout) + t * a.lddo * P::ES;
  for (int j0 = 0; j0 < a.top; j0 += CK) {
    bool ok[CK];
    const char* y[CK];
    char* dy[CK];
    float f[CK], dot[CK];
#pragma unroll
    for (int j = 0; j < CK; ++j) {
      const bool in = j0 + j < a.top;
      const int64_t d = choice_row(in ? a.dest[t * a.top + j0 + j] : -1, a.rows, ok[j]);
      f[j] = in ? a.weights[t * a.top + j0 + j] : 0.0f;
      y[j] = static_cast<const char*>(a.y) + d * a.ldy * P::ES;
      dy[j] = static_cast<char*>(a.dy) + d * a.lddy * P::ES;
      dot[j] = 0.0f;
    }
    for (int64_t c = (int64_t)threadIdx.x * P::VEC; c < a.C; c += 64 * NW * P::VEC) {
      const int n = (int)(a.C - c < P::VEC ? a.C - c : P::VEC);
      const typename P::words g = P::load(dout + c * P::ES, n);
      typename P::words q[CK];
#pragma unroll
      for (int j = 0; j < CK; ++j) q[j] = P::load(y[j] + c * P::ES, n);
      P x;
      x.unpack(g);
#pragma unroll
      for (int j = 0; j < CK; ++j) {
        P u, o;
        u.unpack(q[j]);
#pragma unroll
        for (int i = 0; i < P::VEC; ++i) {
          dot[j] = __builtin_fmaf(x.v[i], u.v[i], dot[j]);
          o.v[i] = f[j] * x.v[i];
        }
        if (ok[j]) P::store(dy[j] + c * P::ES, o.pack(), n);
      }
    }
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    float(*const r)[CK] = red[(j0 / CK) & 1];
#pragma unroll
    for (int j = 0; j < CK; ++j) {
      const float s = group_sum<64>(dot[j]);
      if (NW == 1) dot[j] = s;
      else if (lane == 0) r[w][j] = s;
    }
    if (NW > 1) __syncthreads();
#pragma unroll
    for (int j = 0; j < CK; ++j)
      if (threadIdx.x == j && j0 + j < a.top) {
        float s = dot[j];
        if (NW > 1) {
          s = r[0][j];
#pragma unroll
          for (int i = 1; i < NW; ++i) s = s + r[i][j];
        }
        a.dweights[t * a.top + j0 + j] = ok[j] ? s : 0.0f;
      }
  }
}

struct PieceGrid {
  unsigned wgs;
  uint32_t parts;
  int shift;                              // 6: a wave per 64 pieces of a row
};

// (The caller bounds the waves to 2^31.)
template <int VEC>
PieceGrid piece_grid(int64_t T, int64_t C) {
  const int64_t pieces = (C + VEC - 1) / VEC;
  PieceGrid g{0, 1, 0};
  while (g.shift < 6 && (1 << g.shift) < pieces) ++g.shift;
  int64_t waves;
  if (pieces > 32) {
    g.shift = 6;
    g.parts = (uint32_t)((pieces + 63) / 64);
    waves = T * g.parts;
  } else {
    waves = (T + (64 >> g.shift) - 1) >> (6 - g.shift);
  }
  g.wgs = (unsigned)((waves + 3) / 4);
  return g;
}

template <bool BF16>
hipError_t launch_combine_t(const CombineArgs& a, hipStream_t st) {
  const PieceGrid g = piece_grid<RowPiece<BF16>::VEC>(a.T, a.C);
  if (g.shift == 6) hipLaunchKernelGGL((k_combine<BF16, true>), dim3(g.wgs), dim3(256), 0, st, a, g.parts, g.shift);
  else hipLaunchKernelGGL((k_combine<BF16, false>), dim3(g.wgs), dim3(256), 0, st, a, g.parts, g.shift);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_dispatch_t(const CombineArgs& a, hipStream_t st) {
  const PieceGrid g = piece_grid<RowPiece<BF16>::VEC>(a.T, a.C);
  if (g.shift == 6) hipLaunchKernelGGL((k_dispatch<BF16, true>), dim3(g.wgs), dim3(256), 0, st, a, g.parts, g.shift);
  else hipLaunchKernelGGL((k_dispatch<BF16, false>), dim3(g.wgs), dim3(256), 0, st, a, g.parts, g.shift);
  return hipGetLastError();
}

// About two pieces per lane.
template <bool BF16>
hipError_t launch_backward_t(const CombineArgs& a, hipStream_t st) {
  const int64_t pieces = (a.C + RowPiece<BF16>::VEC - 1) / RowPiece<BF16>::VEC, w = (pieces + 127) / 128;
  const dim3 grid((unsigned)a.T);
  if (w <= 1) hipLaunchKernelGGL((k_combine_backward<BF16, 1>), grid, dim3(64), 0, st, a);
  else if (w <= 2) hipLaunchKernelGGL((k_combine_backward<BF16, 2>), grid, dim3(128), 0, st, a);
  else if (w <= 3) hipLaunchKernelGGL((k_combine_backward<BF16, 3>), grid, dim3(192), 0, st, a);
  else if (w <= 4) hipLaunchKernelGGL((k_combine_backward<BF16, 4>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((k_combine_backward<BF16, 8>), grid, dim3(512), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_combine(const CombineArgs& a, hipStream_t st) {
  return a.bf16 ? launch_combine_t<true>(a, st) : launch_combine_t<false>(a, st);
}
hipError_t launch_dispatch(const CombineArgs& a, hipStream_t st) {
  return a.bf16 ? launch_dispatch_t<true>(a, st) : launch_dispatch_t<false>(a, st);
}
hipError_t launch_combine_backward(const CombineArgs& a, hipStream_t st) {
  return a.bf16 ? launch_backward_t<true>(a, st) : launch_backward_t<false>(a, st);
}

}  // namespace mx
