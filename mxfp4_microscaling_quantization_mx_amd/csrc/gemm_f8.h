// MXFP8 / MXFP6 operands with loads straight to LDS: the 256x256 pipeline of
// the dense and grouped products of any pair of E4M3, E5M2, E2M3, E3M2.
#pragma once

#include "gemm_sched.h"

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

// A buffer offset past the end of any operand: loads there return zeros.
constexpr uint32_t MX_OOB = 0x80000000u;

// 256x256 tiles of 8 waves (4 along M x 2 along N, 64x128 each as 2 x 4
// MFMA tiles) over 128-deep stages: 4 blocks, 128 code bytes per row for an
// FP8 operand (one cache line) and 96 for FP6, and 4 scale bytes.  Each stage
// goes global -> LDS with direct-to-LDS buffer loads into one of two slots
// while the stage in the other slot is multiplied, so the codes never pass
// through VGPRs: per wave and stage, 8 loads of 1 KiB (4 of A, 4 of B: 8
// rows each, a 16-byte chunk per lane; an FP6 row's chunks 6 and 7 read as
// zeros) and one 4-byte scale load (A rows for waves 0-3, B rows for 4-7).
// LDS rows are 128 bytes with XOR-swizzled 16-byte chunks (chunk c of row r
// sits at c ^ ((r >> 1) & 7)), so the operand reads of consecutive rows fall
// in different banks.  The two slots are separate LDS arrays and the stage
// loop is unrolled by two, and the LDS reads are asm blocks that wait only
// for themselves: the compiler would otherwise wait for the loads in flight
// into the other slot before every read.  FP8 lanes read 2 x 16 bytes per
// 64-deep step (K-elements [16 g, 16 g + 16) and [32 + 16 g, 48 + 16 g) of
// the step, g = lane / 32), FP6 lanes 3 x 8 bytes (their whole 24-byte
// block).
namespace f8 {
constexpr int ROWB = 128;                  // LDS bytes per row and stage
constexpr int OPB = 256 * ROWB;            // one operand's stage (32 KiB)
constexpr int SLOT = 2 * OPB;              // A then B
constexpr int SWORDS = 512;                // scale words of a stage: A rows, then B rows
typedef __attribute__((address_space(3))) void* lds_t;
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
template <int F>
constexpr int gbytes() { return elem_bits<F>() == 8 ? 128 : 96; }   // global code bytes of a stage row
}

struct F8Lane {
  __amdgpu_buffer_rsrc_t ra, rb, rs;
  uint32_t va[4], vb[4];                   // code offsets of this lane's 8 loads (stage 0)
  int c[4];                                // their K chunk (16-byte unit of the stage row)
  uint32_t so;                             // scale offset of this lane's row (stage 0)
};

// Issue the loads of stage s into the slot (codes) and sl (scale words).
// Load t of the wave covers rows 8 (4 wave + t) + lane / 8 and puts this
// lane's 16 bytes at LDS chunk lane % 8 of its row, which holds the row's
// K chunk c = (lane % 8) ^ ((row / 2) % 8).  Chunks past the stage row (FP6:
// 6 and 7) or past K read zeros; an FP6 chunk that K ends half-way through
// brings 8 bytes of the next block, whose scale byte compute() clears.
template <int FA, int FB>
__device__ __forceinline__ void f8_issue(const F8Lane& L, int s, int K, uint8_t* slot, uint32_t* sl, int wave) {
  constexpr int RA = f8::gbytes<FA>(), RB = f8::gbytes<FB>();
  const int ka = RA * s, kbb = RB * s;
  const int kbytes_a = K * elem_bits<FA>() / 8, kbytes_b = K * elem_bits<FB>() / 8;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int c16 = 16 * L.c[t];
    const bool ina = c16 < RA && ka + c16 < kbytes_a, inb = c16 < RB && kbb + c16 < kbytes_b;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(L.ra, (f8::lds_t)(slot + 1024 * (4 * wave + t)), 16,
                                             ina ? L.va[t] : MX_OOB, (uint32_t)ka, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(L.rb, (f8::lds_t)(slot + f8::OPB + 1024 * (4 * wave + t)), 16,
                                             inb ? L.vb[t] : MX_OOB, (uint32_t)kbb, 0, 0);
  }
  __builtin_amdgcn_raw_ptr_buffer_load_lds(L.rs, (f8::lds_t)(sl + 64 * wave), 4, L.so, (uint32_t)(4 * s), 0, 0);
}

// This lane's operands of 64-deep step ks for NT row tiles (4096 LDS bytes
// apart) starting at LDS row address `row` (key = the row's chunk swizzle),
// in one asm block that waits for itself only.
template <int F, int NT>
__device__ __forceinline__ void f8_read(uint32_t row, int key, int ks, int hi, v8i out[NT]) {
  if constexpr (elem_bits<F>() == 8) {
    const uint32_t q0 = row + 16 * ((4 * ks + hi) ^ key), q1 = row + 16 * ((4 * ks + 2 + hi) ^ key);
    f8::v4i x[NT], y[NT];
    if constexpr (NT == 2) {
      asm volatile(
          "ds_read_b128 %0, %4\n\t"
          "ds_read_b128 %2, %5\n\t"
          "ds_read_b128 %1, %4 offset:4096\n\t"
          "ds_read_b128 %3, %5 offset:4096\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(y[0]), "=&v"(y[1])
          : "v"(q0), "v"(q1)
          : "memory");
    } else {
      asm volatile(
          "ds_read_b128 %0, %8\n\t"
          "ds_read_b128 %4, %9\n\t"
          "ds_read_b128 %1, %8 offset:4096\n\t"
          "ds_read_b128 %5, %9 offset:4096\n\t"
          "ds_read_b128 %2, %8 offset:8192\n\t"
          "ds_read_b128 %6, %9 offset:8192\n\t"
          "ds_read_b128 %3, %8 offset:12288\n\t"
          "ds_read_b128 %7, %9 offset:12288\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3])
          : "v"(q0), "v"(q1)
          : "memory");
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) out[i] = __builtin_shufflevector(x[i], y[i], 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    // the lane's block: bytes 48 ks + 24 hi + [0, 24) of the stage row, as
    // three 8-byte reads (each inside one 16-byte chunk)
    const int o = 48 * ks + 24 * hi;
    const uint32_t q0 = row + 16 * ((o >> 4) ^ key) + (o & 15);
    const uint32_t q1 = row + 16 * (((o + 8) >> 4) ^ key) + ((o + 8) & 15);
    const uint32_t q2 = row + 16 * (((o + 16) >> 4) ^ key) + ((o + 16) & 15);
    f8::v2i x[NT], y[NT], z[NT];
    if constexpr (NT == 2) {
      asm volatile(
          "ds_read_b64 %0, %6\n\t"
          "ds_read_b64 %2, %7\n\t"
          "ds_read_b64 %4, %8\n\t"
          "ds_read_b64 %1, %6 offset:4096\n\t"
          "ds_read_b64 %3, %7 offset:4096\n\t"
          "ds_read_b64 %5, %8 offset:4096\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(y[0]), "=&v"(y[1]), "=&v"(z[0]), "=&v"(z[1])
          : "v"(q0), "v"(q1), "v"(q2)
          : "memory");
    } else {
      asm volatile(
          "ds_read_b64 %0, %12\n\t"
          "ds_read_b64 %4, %13\n\t"
          "ds_read_b64 %8, %14\n\t"
          "ds_read_b64 %1, %12 offset:4096\n\t"
          "ds_read_b64 %5, %13 offset:4096\n\t"
          "ds_read_b64 %9, %14 offset:4096\n\t"
          "ds_read_b64 %2, %12 offset:8192\n\t"
          "ds_read_b64 %6, %13 offset:8192\n\t"
          "ds_read_b64 %10, %14 offset:8192\n\t"
          "ds_read_b64 %3, %12 offset:12288\n\t"
          "ds_read_b64 %7, %13 offset:12288\n\t"
          "ds_read_b64 %11, %14 offset:12288\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3]),
            "=&v"(z[0]), "=&v"(z[1]), "=&v"(z[2]), "=&v"(z[3])
          : "v"(q0), "v"(q1), "v"(q2)
          : "memory");
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const f8::v4i xy = __builtin_shufflevector(x[i], y[i], 0, 1, 2, 3);
      const f8::v4i zz = {z[i][0], z[i][1], 0, 0};   // an FP6 operand is 6 dwords; the rest zero
      out[i] = __builtin_shufflevector(xy, zz, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
}

// Multiply the stage held in (slot, sl: LDS byte addresses of its codes and
// scale words): 2 steps of 8 MFMAs per wave.  SWAP issues every MFMA with the
// operands (and their formats and scales) exchanged, so that tile (i, j)
// accumulates its transpose: each lane then holds 16 columns of one output
// row, the layout of the quantizing epilogue.
template <int FA, int FB, bool SWAP = false>
__device__ __forceinline__ void f8_compute(v16f acc[2][4], uint32_t slot, uint32_t sl, int s, int K, int wm, int wn,
                                           int l32, int hi) {
  // blocks of this stage below K; the scale bytes of the others (row padding)
  // are cleared to 0, a finite scale: their codes are zero, or for an FP6 row
  // that K ends inside a chunk, 8 bytes whose products with a scale of 2^-127
  // on both sides vanish in float32
  const int nk = (K >> 5) - 4 * s;
  const uint32_t keep = nk >= 4 ? 0xFFFFFFFFu : (1u << (8 * nk)) - 1u;
  // the scale words through an asm read (waiting for itself only)
  const uint32_t wa = sl + 4 * (wm * 64 + l32);
  const uint32_t wb = sl + 4 * (256 + wn * 128 + l32);
  uint32_t q[6];
  asm volatile(
      "ds_read_b32 %0, %6\n\t"
      "ds_read_b32 %1, %6 offset:128\n\t"
      "ds_read_b32 %2, %7\n\t"
      "ds_read_b32 %3, %7 offset:128\n\t"
      "ds_read_b32 %4, %7 offset:256\n\t"
      "ds_read_b32 %5, %7 offset:384\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(q[0]), "=&v"(q[1]), "=&v"(q[2]), "=&v"(q[3]), "=&v"(q[4]), "=&v"(q[5])
      : "v"(wa), "v"(wb)
      : "memory");
  int sa[2], sb[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) sa[i] = (int)((q[i] & keep) >> (8 * hi));
#pragma unroll
  for (int j = 0; j < 4; ++j) sb[j] = (int)((q[2 + j] & keep) >> (8 * hi));
  const int key = (l32 >> 1) & 7;
  const uint32_t ra = slot + (wm * 64 + l32) * f8::ROWB;
  const uint32_t rb = slot + f8::OPB + (wn * 128 + l32) * f8::ROWB;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    v8i a[2], b[4];
    f8_read<FA, 2>(ra, key, ks, hi, a);
    f8_read<FB, 4>(rb, key, ks, hi, b);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (SWAP) {
          if (ks == 0)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[j], a[i], acc[i][j], mfma_fmt<FB>(),
                                                                         mfma_fmt<FA>(), 0, sb[j], 0, sa[i]);
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[j], a[i], acc[i][j], mfma_fmt<FB>(),
                                                                         mfma_fmt<FA>(), 2, sb[j], 2, sa[i]);
        } else {
          if (ks == 0)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[i], b[j], acc[i][j], mfma_fmt<FA>(),
                                                                         mfma_fmt<FB>(), 0, sa[i], 0, sb[j]);
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a[i], b[j], acc[i][j], mfma_fmt<FA>(),
                                                                         mfma_fmt<FB>(), 2, sa[i], 2, sb[j]);
        }
      }
  }
}

// Persistent: one workgroup per CU walks its list of tiles (Sched: the dense
// XCD-contiguous ranges in groups of 8 M-tiles, or the grouped GEMM's expert
// row tiles), and the stage sequence runs on across tiles: the next tile's
// first stage loads into the free slot while the current tile's last stage is
// multiplied and its result stored.
// OUT: 0 float32, 1 bf16, 2 the quantizing epilogue (MXFP4 codes and scale
// bytes along N into qo, from the swapped-operand accumulators), 3 the gated
// block's epilogue (go: forward, or with dH backward; `halves` its row order).
template <int FA, int FB, int OUT, class Sched>
__device__ __forceinline__ void run_f8(const Sched& sc, const MxOperand& A, const MxOperand& B, int K, void* C,
                                       int64_t ldc, int a_2d, int b_2d, uint8_t* slots, uint32_t* sws,
                                       const t256::QOut& qo = t256::QOut{}, const t256c::GateOut* go = nullptr,
                                       int halves = 0) {
  constexpr bool OUT_BF16 = OUT == 1;
  constexpr bool GATED = OUT == 3;
  static_assert(GATED == (Sched::BMAP != t256c::B_ROWS), "the gated epilogue needs the gated row order");
  constexpr bool SWAP = OUT == 2;
  const int ntiles = sc.count();
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l32 = lane & 31, hi = lane >> 5;
  // this lane's K chunks (one per load) and its scale row
  int crow[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int row = 8 * (4 * wave + t) + (lane >> 3);
    crow[t] = (lane & 7) ^ ((row >> 1) & 7);               // the K chunk this lane's LDS chunk holds
  }
  const bool sA = wave < 4;
  const int srow = 64 * (wave & 3) + lane;                    // this lane's scale row within the tile
  const bool s2d = sA ? a_2d != 0 : b_2d != 0;
  const int64_t lds_s = sA ? A.ld_scales : B.ld_scales;
  // Tile j of this workgroup: the lane's load state, and the tile's output
  // origin (row of C, column) and extent.
  auto setup = [&](int j, F8Lane& L, int64_t& crow0, int& n0, int& mlim, int& nlim) {
    const t256::TileInfo ti = sc.tile(j);
    mlim = ti.M - ti.m0;
    nlim = ti.N - ti.n0;
    const int arows = mlim < 256 ? mlim : 256, brows = nlim < 256 ? nlim : 256;
    // row of B for LDS row r, from the tile's first row, or -1 past the end
    // (gated: from the operand's first row, gates and ups in turn)
    auto b_row = [&](int r) {
      if constexpr (!GATED) return r < brows ? r : -1;
      else return halves ? t256c::b_row<t256c::B_HALVES>(ti.n0, ti.N, r)
                         : t256c::b_row<t256c::B_INTERLEAVED>(ti.n0, ti.N, r);
    };
    L.ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(ti.a_codes) + (int64_t)ti.m0 * A.ld_codes, 0,
                                             (uint32_t)(arows * A.ld_codes), 0x00020000);
    L.rb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(ti.b_codes) + (GATED ? 0 : (int64_t)ti.n0 * B.ld_codes), 0,
        (uint32_t)((GATED ? 2 * ti.N : brows) * B.ld_codes), 0x00020000);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int row = 8 * (4 * wave + t) + (lane >> 3);
      L.c[t] = crow[t];
      L.va[t] = row < arows ? (uint32_t)(row * A.ld_codes + 16 * crow[t]) : MX_OOB;
      const int rb = b_row(row);
      L.vb[t] = rb >= 0 ? (uint32_t)(rb * B.ld_codes + 16 * crow[t]) : MX_OOB;
    }
    const int r0 = sA ? ti.m0 : GATED ? 0 : ti.n0;
    const int sr = sA ? (srow < arows ? srow : -1) : b_row(srow);
    const int srows = sA || !GATED ? 256 : 2 * ti.N;
    const uint8_t* sbase = (sA ? ti.a_scales : ti.b_scales) + (int64_t)(s2d ? (r0 >> 5) : r0) * lds_s;
    L.rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(sbase), 0, (uint32_t)((s2d ? srows / 32 : srows) * lds_s),
                                             0x00020000);
    L.so = sr >= 0 ? (uint32_t)((s2d ? (sr >> 5) : sr) * lds_s) : MX_OOB;
    crow0 = ti.c_row0;
    n0 = ti.n0;
  };
  const int nst = (K + 127) / 128;
  const uint32_t a_slots = (uint32_t)(uintptr_t)(f8::lds_t)slots, a_sws = (uint32_t)(uintptr_t)(f8::lds_t)sws;
  F8Lane L;
  int64_t c0 = 0, c0n = 0;
  int n0 = 0, mlim = 0, nlim = 0, n0n = 0, mln = 0, nln = 0;
  if (ntiles > 0) setup(0, L, c0, n0, mlim, nlim);
  if (ntiles > 0 && nst > 0) f8_issue<FA, FB>(L, 0, K, slots, sws, wave);
  int g = 0;                                                  // stages multiplied so far (slot g & 1)
  for (int j = 0; j < ntiles; ++j) {
    t256::Acc acc;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc.t[i][jj][r] = 0.0f;
    for (int s = 0; s < nst; ++s, ++g) {
      // stage s of tile j is in slot g & 1; the other slot takes the next stage
      __builtin_amdgcn_s_waitcnt(0x0F70);      // vmcnt(0): this wave's loads of stage s landed
      __syncthreads();                         // ... every wave's; every wave is done with the other slot
      const int nx = (g + 1) & 1;
      if (s + 1 < nst) {
        f8_issue<FA, FB>(L, s + 1, K, slots + nx * f8::SLOT, sws + nx * f8::SWORDS, wave);
      } else if (j + 1 < ntiles) {
        // tile j issues nothing more: its load state becomes tile j + 1's
        setup(j + 1, L, c0n, n0n, mln, nln);
        f8_issue<FA, FB>(L, 0, K, slots + nx * f8::SLOT, sws + nx * f8::SWORDS, wave);
      }
      f8_compute<FA, FB, SWAP>(acc.t, a_slots + (uint32_t)((g & 1) * f8::SLOT),
                               a_sws + (uint32_t)((g & 1) * 4 * f8::SWORDS), s, K, wm, wn, l32, hi);
    }
    // epilogue: the 256x256 kernels' bounds-checked store path (same wave
    // layout and MFMA tiles), or their quantizing epilogue
    if constexpr (SWAP) {
      t256s::Acc q;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) q.t[i][jj] = acc.t[i][jj];
      t256s::store_tile_mx(q, qo, (int)c0, n0, mlim, nlim);
    } else if constexpr (GATED) {
      const t256c::GateOut q = t256c::load_gate_out(go);
      if (q.dH) {
        if (halves) t256::store_tile_gate<true, t256c::B_HALVES>(acc, q, c0, n0, mlim, nlim);
        else t256::store_tile_gate<true, t256c::B_INTERLEAVED>(acc, q, c0, n0, mlim, nlim);
      } else {
        t256::store_tile_gate<false, t256c::B_INTERLEAVED>(acc, q, c0, n0, mlim, nlim);
      }
    } else {
      constexpr int ES = OUT_BF16 ? 2 : 4;
      t256::store_tile<OUT_BF16>(acc, static_cast<uint8_t*>(C) + (c0 * ldc + n0) * ES, (int)ldc, mlim, nlim);
    }
    if (j + 1 < ntiles) {
      if (nst == 0) setup(j + 1, L, c0n, n0n, mln, nln);
      c0 = c0n;
      n0 = n0n;
      mlim = mln;
      nlim = nln;
    }
  }
}

}  // namespace
}  // namespace mx
