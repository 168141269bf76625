// The gated feed-forward block on MX operands for gfx950: both projections,
// the activation and the product in one kernel, and the backward pass that
// recomputes the projections (formulas in gate_device.h).
//
// The kernels here take any shape, element types, scale layout and alignment;
// large MXFP4 and MXFP8 / MXFP6 problems go to the 256-row pipelines
// (launch_gated).  They run on V_MFMA_SCALE_F32_32X32X64_F8F6F4, 128 K-elements
// of a row at a time; waves that split the K range add their partial tiles
// through LDS in a fixed order.
//  * k_gated_few: 32 rows by 16 hidden columns per workgroup of 8 waves, which
//    split K 8 ways; the B tile is the 32 weight rows of the columns' gates
//    (first 16) and ups (last 16).  For few rows, where reading the weight
//    once with as many loads in flight as possible is all that counts.
//  * k_gated_tile: 128 rows by 64 hidden columns per workgroup of 8 waves (2 x
//    2 of 64 x 32, K split in two), operands staged through LDS; a wave's two B
//    tiles are its columns' gates and ups.
#include "gate_device.h"
#include "mx_device.h"
#include "mx_launch.h"

namespace mx {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// MFMA operand-format field of mx_elem F.
template <int F>
constexpr int mfma_fmt() {
  if constexpr (F == 0) return 4;
  else return ElemT<F>::MFMA;
}

// The expert and rows of row tile `slot` (TM rows each, numbered in expert
// order) from the device offsets, clamped to [0, cap]; every wave works it out
// by itself.  False past the last tile.
template <int TM>
__device__ __forceinline__ bool find_slot(const int32_t* __restrict__ off, int E, int64_t cap, int64_t slot, int& ex,
                                          int64_t& row0, int& rows) {
  const int lane = threadIdx.x & 63;
  int64_t carry = 0;
  for (int base = 0; base < E; base += 64) {
    const int e = base + lane;
    int64_t l0 = 0, h0 = 0;
    if (e < E) {
      l0 = off[e];
      h0 = off[e + 1];
      l0 = l0 < 0 ? 0 : (l0 > cap ? cap : l0);
      h0 = h0 < l0 ? l0 : (h0 > cap ? cap : h0);
    }
    const int tiles = (int)((h0 - l0 + TM - 1) / TM);
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl += v;
    }
    const int64_t s = slot - carry;
    const unsigned long long m = __ballot(s >= incl - tiles && s < incl);
    if (m) {
      const int src = __ffsll((long long)m) - 1;
      const int pre = __shfl(incl - tiles, src, 64);
      const int lo = __shfl((int)l0, src, 64), hi = __shfl((int)h0, src, 64);
      ex = __builtin_amdgcn_readfirstlane(base + src);
      const int r = __builtin_amdgcn_readfirstlane(lo + (int)(s - pre) * TM);
      const int n = __builtin_amdgcn_readfirstlane(hi) - r;
      row0 = r;
      rows = n < TM ? n : TM;
      return true;
    }
    carry += __shfl(incl, 63, 64);
  }
  return false;
}

// One operand row as a lane sees it.
struct OpRow {
  const uint8_t* codes;
  const uint8_t* scales;
};

__device__ __forceinline__ OpRow op_row(const MxOperand& o, int two_d, int64_t row) {
  return {o.codes + row * o.ld_codes, o.scales + (two_d ? row >> 5 : row) * o.ld_scales};
}

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

__device__ __forceinline__ v16f zero16() {
  v16f z;
#pragma unroll
  for (int r = 0; r < 16; ++r) z[r] = 0.0f;
  return z;
}

template <class I>
__device__ __forceinline__ float load_out(const void* p, bool bf16, I i) {
  return bf16 ? bf16lo(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
template <class I>
__device__ __forceinline__ void store_out(void* p, bool bf16, I i, float v) {
  if (bf16) static_cast<uint16_t*>(p)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
  else static_cast<float*>(p)[i] = v;
}

// Row tile `slot` (TM rows) of the problem: its expert, first row and rows.
template <int TM>
__device__ __forceinline__ bool place_slot(const GatedArgs& a, int64_t slot, int& ex, int64_t& row0, int& rows) {
  ex = 0;
  if (a.offsets) return find_slot<TM>(a.offsets, a.E, a.M, slot, ex, row0, rows);
  row0 = slot * TM;
  rows = (int)(a.M - row0 < TM ? a.M - row0 : TM);
  return true;
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

constexpr int FW = 8;               // waves of k_gated_few, splitting K
// Pieces a wave requests before it multiplies the first.  More would cost the
// second workgroup per CU its registers: 64 rows over 32 MXFP8 experts 100 us
// with 2, 145 with 3; MXFP4 53 with 2 or 3, 85 with 4.
constexpr int FD = 2;

template <int FA, int FB>
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
    const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
    if (row < rows && n0 + col < a.N) {
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

// The 16 outputs of one MFMA tile: rows row0 + at + 8 (r / 4) + 4 hi + r % 4
// with at + ... below `rows`, column c.  32-bit offsets from row row0.
template <int ACT>
__device__ __forceinline__ void finish16(const GatedArgs& a, const GateP& p, int64_t row0, int at, int rows, uint32_t c,
                                         int hi, const v16f& g, const v16f& u) {
  if (c >= (uint32_t)a.N) return;
  const int eo = a.out_bf16 ? 2 : 4, eh = a.dh_bf16 ? 2 : 4;
  char* const out = static_cast<char*>(a.out) + row0 * a.ldo * eo;
  const char* const dh = static_cast<const char*>(a.dH) + row0 * a.lddh * eh;
  const uint32_t ld = (uint32_t)a.ldo, ldh = (uint32_t)a.lddh;
  const uint32_t cg = !a.dH || a.halves ? c : 2 * c, cu = a.halves ? (uint32_t)a.N + c : 2 * c + 1;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int row = at + 8 * (r >> 2) + 4 * hi + (r & 3);
    if (row >= rows) continue;
    if (!a.dH) {
      store_out(out, a.out_bf16, row * ld + cg, gate_forward<ACT>(p, g[r], u[r]));
    } else {
      float dg, du;
      gate_backward<ACT>(p, g[r], u[r], load_out(dh, a.dh_bf16, row * ldh + c), dg, du);
      store_out(out, a.out_bf16, row * ld + cg, dg);
      store_out(out, a.out_bf16, row * ld + cu, du);
    }
  }
}

// Rows of one operand of k_gated_tile: 128 rows x 128 K-elements per stage, in
// 16-byte units, staged through registers into LDS by the 256 threads of a K
// half.  Every thread keeps its rows over all stages.
template <int F>
struct TileLoad {
  static constexpr int RB = 16 * elem_bits<F>();      // code bytes of a stage row
  static constexpr int U = RB / 16, N = 128 * U / 256;
  static constexpr int PITCH = RB + 16;               // LDS row pitch: rows start in different banks
  __amdgpu_buffer_rsrc_t r;                           // raw buffer: loads past its end return zeros
  uint32_t off[N];                                    // this thread's units of stage 0
};
constexpr uint32_t PAST = 0xFFFFFF00u;                // an offset past any operand taken here

// One stage of both operands in registers: codes, and the four scale bytes of
// one row (threads 0 .. 127 A rows, 128 .. 255 B rows).
template <int FA, int FB>
struct TileStage {
  uint4 a[TileLoad<FA>::N], b[TileLoad<FB>::N];
  uint32_t sc;
};

// Units of stage d (K-elements 128 d ..); units past the row's end read zeros,
// and of a unit that an FP6 row ends inside only the first half is kept.
template <int F>
__device__ __forceinline__ void fetch_units(const TileLoad<F>& l, uint4 v[TileLoad<F>::N], int d, int kbytes, int tid) {
  using L = TileLoad<F>;
  // (a stage past the row's end adds no scalar offset: the bounds check
  // subtracts it from the buffer's size)
  const uint32_t at = d * L::RB < kbytes ? (uint32_t)(d * L::RB) : 0u;
#pragma unroll
  for (int i = 0; i < L::N; ++i) {
    const int left = kbytes - d * L::RB - 16 * ((tid + 256 * i) % L::U);
    const uint32_t off = left > 0 ? l.off[i] : PAST;
    v[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(l.r, off, at, 0));
    if (F > 2 && left < 16) v[i].z = v[i].w = 0u;
  }
}

template <int F>
__device__ __forceinline__ void put_units(const uint4 v[TileLoad<F>::N], uint8_t* lds, int tid) {
  using L = TileLoad<F>;
#pragma unroll
  for (int i = 0; i < L::N; ++i) {
    const int id = tid + 256 * i, r = id / L::U, u = id % L::U;
    *reinterpret_cast<uint4*>(lds + r * L::PITCH + 16 * u) = v[i];
  }
}

// This lane's operand registers of 64-deep step s from its LDS row.
template <int F>
__device__ __forceinline__ v8i read_units(const uint8_t* row, int s, int hi) {
  if constexpr (elem_bits<F>() == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + 32 * s + 16 * hi);
    return v8i{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
  } else if constexpr (elem_bits<F>() == 8) {
    const uint4 x = *reinterpret_cast<const uint4*>(row + 64 * s + 16 * hi);
    const uint4 y = *reinterpret_cast<const uint4*>(row + 64 * s + 32 + 16 * hi);
    return v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
  } else {
    const uint2* q = reinterpret_cast<const uint2*>(row + 48 * s + 24 * hi);
    const uint2 x = q[0], y = q[1], z = q[2];
    return v8i{(int)x.x, (int)x.y, (int)y.x, (int)y.y, (int)z.x, (int)z.y, 0, 0};
  }
}

// 128 rows by 64 hidden columns.  Waves 0-3 take the first half of the K
// stages and waves 4-7 the second, 2 x 2 waves of 64 rows by 32 columns each;
// LDS row r of B is the gate (r % 64 < 32) or up row of hidden column
// n0 + 32 (r / 64) + r % 32.  Each half has two LDS buffers and holds one more
// stage in registers, or two where both operands are small (HELD): stage s + 1
// is written to LDS and stage s + 1 + HELD requested while stage s is
// multiplied, since with few workgroups the kernel is bound by the latency of
// its loads.
template <int FA, int FB>
__global__ __launch_bounds__(512) void k_gated_tile(GatedArgs a, GateP p, int64_t tiles, int64_t tiles_n, int a_words,
                                                    int b_words) {
  using LA = TileLoad<FA>;
  using LB = TileLoad<FB>;
  constexpr int ABYTES = 128 * LA::PITCH, BBYTES = 128 * LB::PITCH, BUF = ABYTES + BBYTES + 1024;
  constexpr int RED = 8 * 2 * 16 * 64 * 4;
  __shared__ __attribute__((aligned(16))) uint8_t smem[4 * BUF > RED ? 4 * BUF : RED];
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t slot = t / tiles_n;
    const int64_t n0 = (t - slot * tiles_n) * 64;
    if (n0 >= a.N) continue;                          // (columns are padded to 8 tiles)
    int ex, rows;
    int64_t row0;
    if (!place_slot<128>(a, slot, ex, row0, rows)) return;  // past the last tile
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wk = w >> 2, wm = (w >> 1) & 1, wn = w & 1, tid = threadIdx.x & 255;
    const int l32 = lane & 31, hi = lane >> 5;
    MxOperand B = a.B;
    B.codes += ex * a.stride_codes;
    B.scales += ex * a.stride_scales;
    // rows and columns past the end read the last one; their results are dropped
    auto a_row = [&](int r) { return row0 + (r < rows ? r : rows - 1); };
    auto b_row = [&](int r) {
      const int64_t c = n0 + 32 * (r >> 6) + (r & 31), n = c < a.N ? c : a.N - 1;
      const int up = (r >> 5) & 1;
      return a.halves ? up * a.N + n : 2 * n + up;
    };
    LA la;
    LB lb;
    la.r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.A.codes + row0 * a.A.ld_codes), 0,
                                             (uint32_t)(rows * a.A.ld_codes), 0x00020000);
    lb.r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(B.codes), 0, (uint32_t)(2 * a.N * B.ld_codes),
                                             0x00020000);
#pragma unroll
    for (int i = 0; i < LA::N; ++i) {
      const int id = tid + 256 * i;
      la.off[i] = (uint32_t)((a_row(id / LA::U) - row0) * a.A.ld_codes) + 16u * (id % LA::U);
    }
#pragma unroll
    for (int i = 0; i < LB::N; ++i) {
      const int id = tid + 256 * i;
      lb.off[i] = (uint32_t)(b_row(id / LB::U) * B.ld_codes) + 16u * (id % LB::U);
    }
    const bool sa = tid < 128;                        // wave-uniform
    const int64_t sr = sa ? a_row(tid) : b_row(tid - 128);
    const uint8_t* sp = sa ? a.A.scales + (a.a_2d ? sr >> 5 : sr) * a.A.ld_scales
                           : B.scales + (a.b_2d ? sr >> 5 : sr) * B.ld_scales;
    const bool words = sa ? a_words : b_words;
    const int nkb = (int)(a.K / 32), stages = (nkb + 3) / 4, per = (stages + 1) / 2;
    const int abytes = (int)(a.K * elem_bits<FA>() / 8), bbytes = (int)(a.K * elem_bits<FB>() / 8);
    const int d0 = wk * per;                          // stages past the last are zeros at scale 1
    auto fetch = [&](TileStage<FA, FB>& st, int s) {
      const int d = d0 + s;
      fetch_units<FA>(la, st.a, d, abytes, tid);
      fetch_units<FB>(lb, st.b, d, bbytes, tid);
      if (words && 4 * d + 4 <= nkb) {
        st.sc = *reinterpret_cast<const uint32_t*>(sp + 4 * (int64_t)d);
      } else {
        uint32_t v = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) v |= (4 * d + j < nkb ? (uint32_t)sp[4 * (int64_t)d + j] : 127u) << (8 * j);
        st.sc = v;
      }
    };
    uint8_t* const mine = smem + 2 * BUF * wk;
    auto put = [&](const TileStage<FA, FB>& st, int buf) {
      uint8_t* const q = mine + buf * BUF;
      put_units<FA>(st.a, q, tid);
      put_units<FB>(st.b, q + ABYTES, tid);
      reinterpret_cast<uint32_t*>(q + ABYTES + BBYTES)[tid] = st.sc;
    };
    v16f acc[2][2];
    acc[0][0] = acc[0][1] = acc[1][0] = acc[1][1] = zero16();
    auto multiply = [&](int buf) {
      const uint8_t* const q = mine + buf * BUF;
      const uint32_t* const sw = reinterpret_cast<const uint32_t*>(q + ABYTES + BBYTES);
      int xa[2], xb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        xa[i] = (int)(sw[64 * wm + 32 * i + l32] >> (8 * hi));
        xb[i] = (int)(sw[128 + 64 * wn + 32 * i + l32] >> (8 * hi));
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        v8i va[2], vb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          va[i] = read_units<FA>(q + (64 * wm + 32 * i + l32) * LA::PITCH, s, hi);
          vb[i] = read_units<FB>(q + ABYTES + (64 * wn + 32 * i + l32) * LB::PITCH, s, hi);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (s == 0)
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va[i], vb[j], acc[i][j], mfma_fmt<FA>(),
                                                                           mfma_fmt<FB>(), 0, xa[i], 0, xb[j]);
            else
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(va[i], vb[j], acc[i][j], mfma_fmt<FA>(),
                                                                           mfma_fmt<FB>(), 2, xa[i], 2, xb[j]);
          }
      }
    };
    constexpr int HELD = elem_bits<FA>() + elem_bits<FB>() <= 10 ? 2 : 1;
    TileStage<FA, FB> st[HELD];
    if (per > 0) {
      fetch(st[0], 0);
      if (HELD > 1 && per > 1) fetch(st[HELD - 1], 1);
      put(st[0], 0);
      if (per > HELD) fetch(st[0], HELD);
      __syncthreads();
    }
    // stage s + 1 is in st[(s + 1) % HELD]; buffer (s + 1) % 2 was last read in
    // stage s - 1, before the last barrier
    for (int s = 0; s < per; s += 2) {
      if (s + 1 < per) put(st[1 % HELD], 1);
      if (s + 1 + HELD < per) fetch(st[1 % HELD], s + 1 + HELD);
      multiply(0);
      __syncthreads();
      if (s + 1 >= per) break;
      if (s + 2 < per) put(st[0], 0);
      if (s + 2 + HELD < per) fetch(st[0], s + 2 + HELD);
      multiply(1);
      __syncthreads();
    }
    // the two K halves: wave wk finishes row tile wk and hands over the other
    float (*red)[2][16][64] = reinterpret_cast<float (*)[2][16][64]>(smem);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) red[w][j][r][lane] = wk ? acc[0][j][r] : acc[1][j][r];
    __syncthreads();
    v16f gu[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) gu[j][r] = (wk ? acc[1][j][r] : acc[0][j][r]) + red[w ^ 4][j][r][lane];
    const int sub = 64 * wm + 32 * wk;
    const uint32_t col = (uint32_t)n0 + 32 * wn + l32;
    if (p.act == 0) finish16<0>(a, p, row0, sub, rows, col, hi, gu[0], gu[1]);
    else if (p.act == 1) finish16<1>(a, p, row0, sub, rows, col, hi, gu[0], gu[1]);
    else finish16<2>(a, p, row0, sub, rows, col, hi, gu[0], gu[1]);
    __syncthreads();                  // the LDS is free again
  }
}

// Row tiles of TM rows a grouped launch must offer: every expert with rows
// adds at most one partial tile.
int64_t slot_bound(const GatedArgs& a, int TM) {
  if (!a.offsets) return (a.M + TM - 1) / TM;
  return a.M / TM + (a.E < a.M ? a.E : a.M);
}

// Column tiles per row tile, padded to a multiple of 8 where there are several
// row tiles: a column tile's workgroups then run on one XCD (workgroup b on
// XCD b % 8) and share its weight rows in one L2.
int64_t column_tiles(const GatedArgs& a, int TN) {
  const int64_t n = (a.N + TN - 1) / TN;
  return a.M > 32 ? (n + 7) / 8 * 8 : n;
}

unsigned tile_grid(int64_t tiles) { return (unsigned)(tiles < (1 << 20) ? tiles : (1 << 20)); }

template <int FA, int FB>
hipError_t launch_direct(const GatedArgs& a, bool few, hipStream_t st) {
  const GateP p = gate_params(a.act, a.alpha, a.limit, a.up_shift);
  const int a_words = a.A.ld_scales % 4 == 0 && (uintptr_t)a.A.scales % 4 == 0;
  const int b_words = a.B.ld_scales % 4 == 0 && (uintptr_t)a.B.scales % 4 == 0 && a.stride_scales % 4 == 0;
  // k_gated_tile addresses its rows and the weight operand with 32-bit offsets
  const int64_t lim = 0xFFFFFF00ll;
  const bool fits = 128 * a.A.ld_codes < lim && 2 * a.N * a.B.ld_codes < lim && 128 * a.ldo + 2 * a.N < lim / 4 &&
                    128 * a.lddh < lim / 4;
  if (few || !fits) {
    const int64_t tiles_n = column_tiles(a, 16), tiles = tiles_n * slot_bound(a, 32);
    hipLaunchKernelGGL((k_gated_few<FA, FB>), dim3(tile_grid(tiles)), dim3(64 * FW), 0, st, a, p, tiles, tiles_n,
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

// Which kernel (N = K = 2880 unless said; MXFP4, then MXFP8):
//  * k_gated_few while its workgroups are at most 3 per CU: 128 rows 13-16 us
//    against k_gated_tile's 16 (23 / 26), 192 rows 21 / 17 (38 / 26), 1024 rows
//    of 512 x 1024 8.8 / 9.7 (16 / 13).  Grouped, whose weights are read from
//    HBM, up to 8 rows per expert (32 experts, 64 rows 53 us against the
//    pipeline's 68, 256 rows 79 / 78, 512 rows 104 / 83; MXFP8 100 / 140, 137 /
//    147) or 6 workgroups per CU (512 x 1024: 512 rows 11 / 15 us, 1024 rows
//    15 / 15).
//  * k_gated_tile while one workgroup per CU does: 16-18 us (24-28) against the
//    21-24 (44-48) of a pipeline that is not full; with two per CU 33-37
//    (53-57).  Also everything that the pipelines do not take.
//  * the 256-row pipelines beyond.
hipError_t launch_gated(const GatedArgs& a, hipStream_t st) {
  if (a.M == 0 || a.N == 0) return hipSuccess;
  const int64_t cus = cu_count();
  const int64_t few_wgs = (a.N + 15) / 16 * slot_bound(a, 32), tile_wgs = (a.N + 63) / 64 * slot_bound(a, 128);
  const bool few = a.offsets ? a.M <= 8 * (int64_t)a.E || few_wgs <= 6 * cus : few_wgs <= 3 * cus;
  if (!few && (a.offsets || tile_wgs > cus)) {
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
