// Kernels for MX products whose epilogue works on float32 accumulators, at any
// shape, element types, scale layout and alignment: bodies shared by the gated
// block (gated.hip) and the linear layer with an epilogue (linear.hip).
//
// They run on V_MFMA_SCALE_F32_32X32X64_F8F6F4, 128 K-elements of a row at a
// time.  LIN: the B tile's rows are consecutive rows of the weight, each an
// output column; otherwise they are the gates and ups of half as many hidden
// columns (a.N counts columns in both).
#pragma once

#include "gate_device.h"
#include "group_device.h"
#include "launch_rule.h"
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

constexpr uint32_t PAST = 0x80000000u;           // a buffer offset past any operand (taken below 2 GiB)

// One operand row as a lane sees it.
struct OpRow {
  const uint8_t* codes;
  const uint8_t* scales;
};

__device__ __forceinline__ OpRow op_row(const MxOperand& o, int two_d, int64_t row) {
  return {o.codes + row * o.ld_codes, o.scales + (two_d ? row >> 5 : row) * o.ld_scales};
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

// One output of the linear layer from its sum of products (bias of expert ex).
template <int ACT>
__device__ __forceinline__ float linear_value(const GateP& p, bool backward, float x, float r) {
  float d;
  if constexpr (ACT == 3) return x + r;
  else if (backward) return gate_act<ACT, true>(p, x, d), r * d;
  else return gate_act<ACT, false>(p, x, d) + r;
}
__device__ __forceinline__ float linear_out(const LinearArgs& a, const GateP& p, float x, float r) {
  if (p.act == 0) return linear_value<0>(p, a.backward, x, r);
  if (p.act == 1) return linear_value<1>(p, a.backward, x, r);
  if (p.act == 2) return linear_value<2>(p, a.backward, x, r);
  return linear_value<3>(p, a.backward, x, r);
}
__device__ __forceinline__ float linear_bias(const LinearArgs& a, int ex, int64_t c) {
  return a.bias ? load_out(a.bias, a.bias_bf16, ex * a.bias_stride + c) : 0.0f;
}

// Rows of the weight operand.
template <bool LIN>
__host__ __device__ __forceinline__ int64_t weight_rows(const GatedArgs& a) { return LIN ? a.N : 2 * a.N; }

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

// The outputs of two MFMA tiles of the linear layer side by side: rows as above, columns
// c and c + 32, x their sums of products.  Every element is loaded and stored through
// bounds-checked buffers, all of them requested before the first is used and with no
// choice between them (a type chosen per element makes 32 waits: 34 us for 25 at 1037 x
// 1451 x 2912).
template <int ACT>
__device__ __forceinline__ void finish_linear(const LinearArgs& a, const GateP& p, int64_t row0, int at, int rows,
                                              uint32_t c, int ex, int hi, const v16f x[2]) {
  auto rsrc = [&](const void* base, int64_t ld, int es) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(base)) + row0 * ld * es, 0,
                                             (uint32_t)(((rows - 1) * ld + a.N) * es), 0x00020000);
  };
  const uint32_t first = (uint32_t)(at + 4 * hi);
  // (rows past the tile's lie past its buffer, which ends with its last row)
  auto offset = [&](int j, int r, uint32_t ld, int es) {
    const uint32_t row = first + 8 * (r >> 2) + (r & 3);
    return c + 32 * j < (uint32_t)a.N ? (row * ld + c + 32 * j) * es : PAST;
  };
  uint32_t w[2][16];
  float b[2] = {0.0f, 0.0f};
  if (a.bias) {
#pragma unroll
    for (int j = 0; j < 2; ++j) b[j] = linear_bias(a, ex, c + 32 * j < (uint32_t)a.N ? c + 32 * j : a.N - 1);
  }
  const uint32_t ldr = (uint32_t)a.lddh, ldo = (uint32_t)a.ldo;
  if (!a.dH) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) w[j][r] = 0u;
  } else if (a.dh_bf16) {
    const __amdgpu_buffer_rsrc_t rr = rsrc(a.dH, a.lddh, 2);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        w[j][r] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(rr, offset(j, r, ldr, 2), 0, 0)
                  << 16;
  } else {
    const __amdgpu_buffer_rsrc_t rr = rsrc(a.dH, a.lddh, 4);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        w[j][r] = __builtin_amdgcn_raw_buffer_load_b32(rr, offset(j, r, ldr, 4), 0, 0);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      w[j][r] = __float_as_uint(linear_value<ACT>(p, a.backward, x[j][r] + b[j], __uint_as_float(w[j][r])));
  if (a.out_bf16) {
    const __amdgpu_buffer_rsrc_t ro = rsrc(a.out, a.ldo, 2);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, (__bf16)__uint_as_float(w[j][r])), ro,
                                              offset(j, r, ldo, 2), 0, 0);
  } else {
    const __amdgpu_buffer_rsrc_t ro = rsrc(a.out, a.ldo, 4);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        __builtin_amdgcn_raw_buffer_store_b32(w[j][r], ro, offset(j, r, ldo, 4), 0, 0);
  }
}

// ---------------------------------------------------------------- 128 x 128 tiles
// A stage is 128 K-elements of the tile's 128 rows of A and 128 of B: LDS row
// r of B is weight row n0 + r, or the gate (r % 64 < 32) or up row of hidden column
// n0 + 32 (r / 64) + r % 32.  Codes and scale words go straight from global memory to LDS, into
// one of RING slots, RING - 1 stages ahead of the one multiplied: with one
// workgroup per CU nothing else hides the latency of the loads.  Waves 0-3
// multiply the first 64 elements of every stage and waves 4-7 the rest, 2 x 2
// waves of 64 rows by 32 columns each, and add their sums at the end: 64 KiB of
// LDS reads per stage in MXFP8, where 8 waves of 32 x 32 read 96 (21.9 us
// against 22.7).  One barrier per stage.  LDS rows hold the stage's codes in
// 16-byte chunks, XOR-swizzled so that 16 consecutive rows reading one chunk
// hit different banks.
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));

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

template <bool LIN, int FA, int FB, class Args>
__device__ __forceinline__ void row_tiles(const Args& a, const GateP& p, int64_t tiles, int64_t tiles_n, int a_words,
                                          int b_words) {
  constexpr int TN = LIN ? 128 : 64;                  // columns
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
    const int n0 = (int)(t - slot * tiles_n) * TN;
    if (n0 >= a.N) continue;                          // (columns are padded to 8 tiles)
    int ex, rows;
    int64_t row0;
    if (!place_slot<128>(a, slot, ex, row0, rows)) return;  // past the last tile
    const uint8_t* const bc = a.B.codes + ex * a.stride_codes;
    const uint8_t* const bs = a.B.scales + ex * a.stride_scales;
    // rows and columns past the end read the last one; their results are dropped
    auto a_row = [&](int r) { return r < rows ? r : rows - 1; };
    auto b_row = [&](int r) {
      if constexpr (LIN) {
        return n0 + r < a.N ? n0 + r : (int)a.N - 1;
      } else {
        const int c = n0 + 32 * (r >> 6) + (r & 31), n = c < a.N ? c : (int)a.N - 1, up = (r >> 5) & 1;
        return a.halves ? up * (int)a.N + n : 2 * n + up;
      }
    };
    TileLoads<FA> la;
    TileLoads<FB> lb;
    la.r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.A.codes + row0 * a.A.ld_codes), 0,
                                             (uint32_t)(rows * a.A.ld_codes), 0x00020000);
    lb.r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(bc), 0, (uint32_t)(weight_rows<LIN>(a) * a.B.ld_codes),
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
    const int64_t sfirst = s2 ? s0 >> 5 : s0, slast = s2 ? (s0 + (sa ? rows : weight_rows<LIN>(a)) - 1) >> 5
                                                         : s0 + (sa ? rows : weight_rows<LIN>(a)) - 1;
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
    if constexpr (LIN) {
      const uint32_t c = (uint32_t)n0 + 64 * wn + l32;
      if (p.act == 0) finish_linear<0>(a, p, row0, sub, rows, c, ex, hi, gu);
      else if (p.act == 1) finish_linear<1>(a, p, row0, sub, rows, c, ex, hi, gu);
      else if (p.act == 2) finish_linear<2>(a, p, row0, sub, rows, c, ex, hi, gu);
      else finish_linear<3>(a, p, row0, sub, rows, c, ex, hi, gu);
      __syncthreads();                // the LDS is free again
      continue;
    }
    const uint32_t col = (uint32_t)n0 + 32 * wn + l32;
    if (p.act == 0) finish16<0>(a, p, row0, sub, rows, col, hi, gu[0], gu[1]);
    else if (p.act == 1) finish16<1>(a, p, row0, sub, rows, col, hi, gu[0], gu[1]);
    else finish16<2>(a, p, row0, sub, rows, col, hi, gu[0], gu[1]);
    __syncthreads();                  // the LDS is free again
  }
}

int64_t slot_bound(const GatedArgs& a, int TM) { return row_tiles_bound(a.M, a.offsets ? a.E : 0, TM); }

unsigned tile_grid(int64_t tiles) { return (unsigned)(tiles < (1 << 20) ? tiles : (1 << 20)); }

// Whether 32-bit offsets reach a tile's rows, the weight operand and the buffers
// (row_tiles needs it).
template <bool LIN>
bool row_tiles_fit(const GatedArgs& a) {
  const int64_t lim = 1ll << 31, nb = weight_rows<LIN>(a);
  return 128 * a.A.ld_codes < lim && nb * a.B.ld_codes < lim && 128 * a.A.ld_scales < lim && nb * a.B.ld_scales < lim &&
         128 * a.ldo + 2 * a.N < lim / 4 && 128 * a.lddh < lim / 4;
}

struct Words { int a, b; };               // scale rows are 4-byte aligned
Words scale_words(const GatedArgs& a) {
  return {a.A.ld_scales % 4 == 0 && (uintptr_t)a.A.scales % 4 == 0,
          a.B.ld_scales % 4 == 0 && (uintptr_t)a.B.scales % 4 == 0 && a.stride_scales % 4 == 0};
}

}  // namespace
}  // namespace mx
