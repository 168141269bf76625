// The gated feed-forward block on MX operands for gfx950: both projections,
// the activation and the product in one kernel, and the backward pass that
// recomputes the projections (formulas in gate_device.h).
//
// The kernels here take any shape, element types, scale layout and alignment;
// large MXFP4 and MXFP8 / MXFP6 problems go to the 256-row pipelines
// (launch_gated).  They run on V_MFMA_SCALE_F32_32X32X64_F8F6F4, 128 K-elements
// of a row at a time; waves that split the K range add their partial tiles
// through LDS in a fixed order.
//  * k_gated_few: 32 rows by 16 hidden columns per workgroup of 8 or 2 waves,
//    which split K; the B tile is the 32 weight rows of the columns' gates
//    (first 16) and ups (last 16).  For few rows, where reading the weight
//    once with as many loads in flight as possible is all that counts.
//  * k_gated_tile: 128 rows by 64 hidden columns per workgroup of 8 waves,
//    operands staged through a ring in LDS; a wave's two B tiles are its
//    columns' gates and ups.
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

// ---------------------------------------------------------------- 128 rows x 64 columns
// A stage is 128 K-elements of the tile's 128 rows of A and 128 of B: LDS row
// r of B is the gate (r % 64 < 32) or up row of hidden column n0 + 32 (r / 64)
// + r % 32.  Codes and scale words go straight from global memory to LDS, into
// one of RING slots, RING - 1 stages ahead of the one multiplied: with one
// workgroup per CU nothing else hides the latency of the loads.  Waves 0-3
// multiply the first 64 elements of every stage and waves 4-7 the rest, 2 x 2
// waves of 64 rows by 32 columns each, and add their sums at the end: 64 KiB of
// LDS reads per stage in MXFP8, where 8 waves of 32 x 32 read 96 (21.9 us
// against 22.7).  One barrier per stage.  LDS rows hold the stage's codes in
// 16-byte chunks, XOR-swizzled so that 16 consecutive rows reading one chunk
// hit different banks.
//
// 512 x 2880 x 2880: MXFP4 17.8 us, MXFP8 23.4, of which 7.5 are the launch, the
// first loads and the epilogue, and the rest 0.41 and 0.67 us per stage: 10 and
// 12 TB/s out of the XCDs' L2s, which a larger tile would lower and leave CUs
// idle for.  Staged through registers with two LDS buffers: 18.9 and 28.2.
// RING 3 or 5 (with a remainder to take per stage) costs MXFP4 1 us, MXFP8
// none; 8 slots MXFP4 1 us.
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
constexpr uint32_t PAST = 0x80000000u;           // a buffer offset past any operand (taken below 2 GiB)

template <int F>
struct TileOp {
  static constexpr int RB = 16 * elem_bits<F>(); // code bytes of a stage row (64, 96 or 128)
  static constexpr int PITCH = F == 0 ? 64 : 128;
  static constexpr int CH = PITCH / 16;          // chunks of an LDS row
  static constexpr int LOADS = 128 * CH / 512;   // 1 KiB loads per wave and stage
  static constexpr int BYTES = 128 * PITCH;
  static __device__ __forceinline__ int key(int row) { return F == 0 ? (row >> 2) & 3 : (row >> 1) & 7; }
};

template <int FA, int FB>
struct TileSlot {
  static constexpr int SCALES = TileOp<FA>::BYTES + TileOp<FB>::BYTES;   // per wave 64 words, the first 32 rows'
  static constexpr int BYTES = SCALES + 2048;
  static constexpr int RING = 4;                 // (a power of two: the slot of a stage is a mask)
  static constexpr int LOADS = TileOp<FA>::LOADS + TileOp<FB>::LOADS + 1;
};

// One load of a wave straight into LDS: 16 or 4 bytes per lane, at dst + 16 or
// 4 times the lane.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t off, uint32_t so) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)dst, 16, off, so, 0, 0);
}
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t off, uint32_t so) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)dst, 4, off, so, 0, 0);
}

// LDS row of lane `lane` of load i of wave `wave`.
template <int F>
__device__ __forceinline__ int tile_row(int wave, int lane, int i) {
  return (64 / TileOp<F>::CH) * (wave * TileOp<F>::LOADS + i) + lane / TileOp<F>::CH;
}

// One operand's loads of this wave: per load the row's offset and its chunk.
template <int F>
struct TileLoads {
  using O = TileOp<F>;
  __amdgpu_buffer_rsrc_t r;
  uint32_t row[O::LOADS];
  int chunk[O::LOADS];

  // Request stage d into LDS at dst.  Chunks past the stage row or the row's
  // end read zeros; a stage past the row's end adds no scalar offset (the
  // bounds check subtracts it from the buffer's size).
  __device__ __forceinline__ void issue(int d, int kbytes, uint8_t* dst, int wave) const {
    const int at = d * O::RB;
    const uint32_t so = at < kbytes ? (uint32_t)at : 0u;
#pragma unroll
    for (int i = 0; i < O::LOADS; ++i) {
      const int c16 = 16 * chunk[i];
      const bool live = c16 < O::RB && at + c16 < kbytes;
      load_lds16(r, dst + 1024 * (wave * O::LOADS + i), live ? row[i] + c16 : PAST, so);
    }
  }
};

// The operand registers of 64-deep step `step` for this lane's rows of two row
// tiles (LDS addresses `row` and 32 rows on) and their scale words (LDS
// addresses sc and 64 words on), in one asm block that waits for itself only
// (the compiler would wait for every load in flight).
template <int F>
__device__ __forceinline__ void tile_read(uint32_t row, int key, int hi, int step, uint32_t sc, v8i out[2],
                                          uint32_t sw[2]) {
  if constexpr (elem_bits<F>() == 4) {
    v4i x, y;
    asm volatile(
        "ds_read_b32 %2, %5\n\tds_read_b32 %3, %5 offset:256\n\t"
        "ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:2048\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(x), "=&v"(y), "=&v"(sw[0]), "=&v"(sw[1])
        : "v"(row + 16 * ((2 * step + hi) ^ key)), "v"(sc)
        : "memory");
    out[0] = v8i{x[0], x[1], x[2], x[3], 0, 0, 0, 0};
    out[1] = v8i{y[0], y[1], y[2], y[3], 0, 0, 0, 0};
  } else if constexpr (elem_bits<F>() == 8) {
    v4i x[4];
    asm volatile(
        "ds_read_b32 %4, %8\n\tds_read_b32 %5, %8 offset:256\n\t"
        "ds_read_b128 %0, %6\n\tds_read_b128 %1, %7\n\t"
        "ds_read_b128 %2, %6 offset:4096\n\tds_read_b128 %3, %7 offset:4096\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(sw[0]), "=&v"(sw[1])
        : "v"(row + 16 * ((4 * step + hi) ^ key)), "v"(row + 16 * ((4 * step + 2 + hi) ^ key)), "v"(sc)
        : "memory");
#pragma unroll
    for (int t = 0; t < 2; ++t) out[t] = __builtin_shufflevector(x[2 * t], x[2 * t + 1], 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    // the lane's 24-byte block, as 8-byte reads inside chunks
    uint32_t at[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int o = 48 * step + 24 * hi + 8 * k;
      at[k] = row + 16 * ((o >> 4) ^ key) + (o & 15);
    }
    v2i x[6];
    asm volatile(
        "ds_read_b32 %6, %11\n\tds_read_b32 %7, %11 offset:256\n\t"
        "ds_read_b64 %0, %8\n\tds_read_b64 %1, %9\n\tds_read_b64 %2, %10\n\tds_read_b64 %3, %8 offset:4096\n\t"
        "ds_read_b64 %4, %9 offset:4096\n\tds_read_b64 %5, %10 offset:4096\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(x[4]), "=&v"(x[5]), "=&v"(sw[0]), "=&v"(sw[1])
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(sc)
        : "memory");
#pragma unroll
    for (int t = 0; t < 2; ++t)
      out[t] = v8i{x[3 * t][0], x[3 * t][1], x[3 * t + 1][0], x[3 * t + 1][1], x[3 * t + 2][0], x[3 * t + 2][1], 0, 0};
  }
}

template <int FA, int FB>
__global__ __launch_bounds__(512) void k_gated_tile(GatedArgs a, GateP p, int64_t tiles, int64_t tiles_n, int a_words,
                                                    int b_words) {
  using OA = TileOp<FA>;
  using OB = TileOp<FB>;
  using SL = TileSlot<FA, FB>;
  static_assert(SL::RING * SL::BYTES >= 8 * 2 * 16 * 64 * 4, "the K halves are added through the ring's LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[SL::RING * SL::BYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wave >> 2, wm = (wave >> 1) & 1, wn = wave & 1, l32 = lane & 31, hi = lane >> 5;
  const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr)lds;
  const int nkb = (int)(a.K / 32), stages = (nkb + 3) / 4;
  const int abytes = (int)(a.K * elem_bits<FA>() / 8), bbytes = (int)(a.K * elem_bits<FB>() / 8);
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t slot = t / tiles_n;
    const int n0 = (int)(t - slot * tiles_n) * 64;
    if (n0 >= a.N) continue;                          // (columns are padded to 8 tiles)
    int ex, rows;
    int64_t row0;
    if (!place_slot<128>(a, slot, ex, row0, rows)) return;  // past the last tile
    const uint8_t* const bc = a.B.codes + ex * a.stride_codes;
    const uint8_t* const bs = a.B.scales + ex * a.stride_scales;
    // rows and columns past the end read the last one; their results are dropped
    auto a_row = [&](int r) { return r < rows ? r : rows - 1; };
    auto b_row = [&](int r) {
      const int c = n0 + 32 * (r >> 6) + (r & 31), n = c < a.N ? c : (int)a.N - 1, up = (r >> 5) & 1;
      return a.halves ? up * (int)a.N + n : 2 * n + up;
    };
    TileLoads<FA> la;
    TileLoads<FB> lb;
    la.r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.A.codes + row0 * a.A.ld_codes), 0,
                                             (uint32_t)(rows * a.A.ld_codes), 0x00020000);
    lb.r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(bc), 0, (uint32_t)(2 * a.N * a.B.ld_codes),
                                             0x00020000);
#pragma unroll
    for (int i = 0; i < OA::LOADS; ++i) {
      const int r = tile_row<FA>(wave, lane, i);
      la.row[i] = (uint32_t)(a_row(r) * (int)a.A.ld_codes);
      la.chunk[i] = (lane % OA::CH) ^ OA::key(r);
    }
#pragma unroll
    for (int i = 0; i < OB::LOADS; ++i) {
      const int r = tile_row<FB>(wave, lane, i);
      lb.row[i] = (uint32_t)(b_row(r) * (int)a.B.ld_codes);
      lb.chunk[i] = (lane % OB::CH) ^ OB::key(r);
    }
    // scale words: waves 0-3 32 rows of A each, 4-7 of B, in the lower half-wave
    const bool sa = wave < 4;
    const int sr = sa ? a_row(32 * wave + l32) : b_row(32 * (wave - 4) + l32);
    const int64_t s0 = sa ? row0 : 0;                 // (A's rows count from row0)
    const bool s2 = sa ? a.a_2d : a.b_2d;
    const int64_t sld = sa ? a.A.ld_scales : a.B.ld_scales;
    const int64_t sfirst = s2 ? s0 >> 5 : s0, slast = s2 ? (s0 + (sa ? rows : 2 * a.N) - 1) >> 5
                                                         : s0 + (sa ? rows : 2 * a.N) - 1;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>((sa ? a.A.scales : bs) + sfirst * sld), 0, (uint32_t)((slast - sfirst + 1) * sld),
        0x00020000);
    const int64_t srow = s2 ? ((s0 + sr) >> 5) - sfirst : sr;
    const uint32_t soff = hi ? PAST : (uint32_t)(srow * sld);
    auto issue = [&](int d) {
      uint8_t* const q = lds + (d % SL::RING) * SL::BYTES;
      la.issue(d, abytes, q, wave);
      lb.issue(d, bbytes, q + OA::BYTES, wave);
      const bool in = d < stages;
      if (sa ? a_words : b_words) {
        load_lds4(rs, q + SL::SCALES + 256 * wave, in ? soff : PAST, in ? 4u * d : 0u);
      } else {                        // rows that do not start at a word: bytes, waiting for every load
        uint32_t v = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rs, 4 * d + j < nkb ? soff + 4 * d + j : PAST, 0, 0)
               << (8 * j);
        *reinterpret_cast<uint32_t*>(q + SL::SCALES + 256 * wave + 4 * lane) = v;
      }
    };
    v16f acc[2][2];
    acc[0][0] = acc[0][1] = acc[1][0] = acc[1][1] = zero16();
    if (stages > 0)
#pragma unroll 1
      for (int d = 0; d < SL::RING - 1; ++d) issue(d);
    for (int s = 0; s < stages; ++s) {
      // this wave's loads of stage s landed (and its own writes to LDS; those of
      // the RING - 2 stages after it may be on their way), then every wave's; and
      // every wave is done with stage s - 1, whose slot takes stage s + RING - 1
      constexpr int N = (SL::RING - 2) * SL::LOADS;
      static_assert(N <= 63, "the counter has 6 bits");
      __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4));
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      issue(s + SL::RING - 1);
      const uint32_t q = base + (uint32_t)((s % SL::RING) * SL::BYTES);
      const int ra = 64 * wm + l32, rb = 64 * wn + l32;
      uint32_t xa[2], xb[2];
      v8i va[2], vb[2];
      tile_read<FA>(q + ra * OA::PITCH, OA::key(ra), hi, wk, q + SL::SCALES + 512 * wm + 4 * l32, va, xa);
      tile_read<FB>(q + OA::BYTES + rb * OB::PITCH, OB::key(rb), hi, wk, q + SL::SCALES + 1024 + 512 * wn + 4 * l32, vb,
                    xb);
      // scale bytes of blocks past K become 0, a finite scale: their codes are
      // zero, or 8 bytes of an FP6 row's padding that vanish at 2^-127 squared
      const int kb = 2 * wk + hi;
      const uint32_t keep = 4 * s + kb < nkb ? 0xFFu : 0u;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              va[i], vb[j], acc[i][j], mfma_fmt<FA>(), mfma_fmt<FB>(), 0, (int)((xa[i] >> (8 * kb)) & keep), 0,
              (int)((xb[j] >> (8 * kb)) & keep));
    }
    __builtin_amdgcn_s_waitcnt(0x0070);               // the loads past the last stage write zeros
    __syncthreads();
    // the two K halves: wave wk finishes row tile wk and hands over the other
    float (*red)[2][16][64] = reinterpret_cast<float (*)[2][16][64]>(lds);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) red[wave][j][r][lane] = wk ? acc[0][j][r] : acc[1][j][r];
    __syncthreads();
    v16f gu[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) gu[j][r] = (wk ? acc[1][j][r] : acc[0][j][r]) + red[wave ^ 4][j][r][lane];
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
  const int64_t lim = 1ll << 31;
  const bool fits = 128 * a.A.ld_codes < lim && 2 * a.N * a.B.ld_codes < lim &&
                    128 * a.A.ld_scales < lim && 2 * a.N * a.B.ld_scales < lim && 128 * a.ldo + 2 * a.N < lim / 4 &&
                    128 * a.lddh < lim / 4;
  if (few || !fits) {
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
