// The gated block on the 256x256 MXFP4 pipeline (gemm_tile256.h): a tile is
// 256 rows by 128 hidden columns, its 256 B rows the gates and ups of those
// columns, and the epilogue applies the block's formula (forward) or its
// derivative (backward) to the accumulators, so the projections never reach
// memory in either direction.
//
// The B rows of a tile are taken in the order that gives each wave's four MFMA
// column tiles as gate, gate, up, up of the same 64 hidden columns: a gate and
// its up then sit in one lane's accumulators.
//
// Forward 16384 x 2880 x 2880: 151-155 us, 3.5-3.6 PFLOP/s; the plain product of
// the same operands with bf16 output takes 174 on the same card, its epilogue
// writing twice the bytes.  The MFMA pipeline bounds it: 123 us with no
// epilogue at all.  Backward: 201-204 us, 316 MB moved; without its stores 35 us
// less, without the reads of dH 28, without the derivatives 24, without all
// three 127 (of 208 then).  What remains of the epilogue is not hidden since one workgroup
// fills a CU's registers and all reach their tile ends together; starting the
// workgroups in 2 to 8 phases changed nothing, nor did bringing dH into L2 a
// stage ahead, nor loading the next tile's second stage before the stores.
// Grouped, 65536 rows over 32 experts: 634-654 us, 3.3-3.4 PFLOP/s; backward of
// 16384 rows over 32 experts 260-291, of which ragged row tiles take a quarter
// (80 row tiles of 256 for 64 full ones' rows); its kernels spill 10-11 VGPRs
// (44-52 bytes of scratch per lane; the dense ones 3-5, forward none).
#define MX_T256_NS t256
#define MX_T256_SWAP 0
#include "gemm_tile256.h"
#undef MX_T256_NS
#undef MX_T256_SWAP
#include "gemm_sched.h"
#include "mx_device.h"
#include "mx_launch.h"

namespace mx {
namespace {

template <bool A2D, bool B2D, int BMAP, bool BWD>
__global__ __launch_bounds__(64 * GW, 1) void k_gated256(MxOperand A, MxOperand B, int M, int N, int K,
                                                         t256c::GateOut go, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[t256::LDS_BYTES];
  __shared__ t256c::GateOut sgo;
  if (threadIdx.x == 0) sgo = go;
  __syncthreads();
  const DenseSchedT<BMAP> sc{A.codes, A.scales, B.codes, B.scales, M, N, tiles_m, tiles_n,
                             XcdShare((int)blockIdx.x, (int)gridDim.x, tiles_m * tiles_n)};
  const t256::Strides sd{(int)A.ld_codes, (int)A.ld_scales, (int)B.ld_codes, (int)B.ld_scales};
  t256::run_tiles<A2D, B2D, BWD ? t256::OUT_GATE_BWD : t256::OUT_GATE, true>(sc, sd, K, nullptr, 0, lds, t256::QOut{},
                                                                            &sgo);
}

template <bool B2D, int BMAP, bool BWD>
__global__ __launch_bounds__(64 * GW, 1) void k_grouped_gated256(MxOperand A, MxOperand B, int64_t M_cap, int N,
                                                                 int K, const int32_t* __restrict__ offsets, int E,
                                                                 int64_t stride_codes, int64_t stride_scales,
                                                                 t256c::GateOut go, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[t256::LDS_BYTES];
  __shared__ int tab[3 * GG_EMAX + 1];
  __shared__ GroupedParams prm;
  __shared__ t256c::GateOut sgo;
  build_expert_table(offsets, E, M_cap, tab);   // ends with a barrier
  const int total_slots = tab[E];
  if (threadIdx.x == 0) {
    prm = GroupedParams{A.codes, A.scales, B.codes, B.scales, stride_codes, stride_scales, (int)A.ld_codes,
                        (int)A.ld_scales, N, tiles_n, E, total_slots, 0, 0};
    sgo = go;
  }
  __syncthreads();
  const GroupedSchedT<BMAP> sc{&prm, tab, XcdShare((int)blockIdx.x, (int)gridDim.x, total_slots * tiles_n)};
  const t256::Strides sd{(int)A.ld_codes, (int)A.ld_scales, (int)B.ld_codes, (int)B.ld_scales};
  t256::run_tiles<false, B2D, BWD ? t256::OUT_GATE_BWD : t256::OUT_GATE, true>(sc, sd, K, nullptr, 0, lds,
                                                                              t256::QOut{}, &sgo);
}

}  // namespace

// The pipeline fetches scale rows 16 bytes at a time and addresses an operand,
// and a tile's rows of the buffers, with 32-bit offsets.
bool gated256_layout_ok(const GatedArgs& a) {
  const int64_t lim = 1ll << 31;
  const bool words = a.A.ld_scales % 16 == 0 && a.B.ld_scales % 16 == 0 && a.stride_scales % 16 == 0 &&
                     (uintptr_t)a.A.scales % 16 == 0 && (uintptr_t)a.B.scales % 16 == 0;
  const int64_t arows = a.offsets ? 256 : a.M;
  const bool small = arows * a.A.ld_codes < lim && 2 * a.N * a.B.ld_codes < lim && arows * a.A.ld_scales < lim &&
                     2 * a.N * a.B.ld_scales < lim && 256 * a.ldo * 4 < lim && 256 * a.lddh * 4 < lim &&
                     a.K < (1ll << 30);
  const int64_t slots = a.offsets ? (a.M + 255) / 256 + a.E : (a.M + 255) / 256;
  return a.a_elem == 0 && a.b_elem == 0 && words && small && (!a.offsets || a.E <= GG_EMAX) &&
         slots * ((a.N + 127) / 128) < lim;
}

hipError_t launch_gated256(const GatedArgs& a, hipStream_t st) {
  const int cus = cu_count();
  const int tiles_n = (int)((a.N + 127) / 128);
  const int64_t tiles_m = a.offsets ? (a.M + 255) / 256 + a.E : (a.M + 255) / 256;
  const int64_t tiles = tiles_m * tiles_n;
  const unsigned nwg = (unsigned)(tiles < cus ? tiles : cus);
  const t256c::GateOut go{gate_params(a.act, a.alpha, a.limit, a.up_shift), a.out, a.dH, (int)a.ldo, (int)a.lddh,
                          (int)a.out_bf16, (int)a.dh_bf16};
#define MX_GT(A_, B_, L_, D_)                                                                                       \
  do {                                                                                                              \
    if (a.offsets) {                                                                                                \
      if constexpr (!(A_))                                                                                          \
        hipLaunchKernelGGL((k_grouped_gated256<B_, L_, D_>), dim3(nwg), dim3(64 * GW), 0, st, a.A, a.B, a.M,        \
                           (int)a.N, (int)a.K, a.offsets, a.E, a.stride_codes, a.stride_scales, go, tiles_n);       \
    } else {                                                                                                        \
      hipLaunchKernelGGL((k_gated256<A_, B_, L_, D_>), dim3(nwg), dim3(64 * GW), 0, st, a.A, a.B, (int)a.M,         \
                         (int)a.N, (int)a.K, go, (int)tiles_m, tiles_n);                                            \
    }                                                                                                               \
  } while (0)
#define MX_GT_D(A_, B_, L_) \
  if (a.dH) MX_GT(A_, B_, L_, true); else MX_GT(A_, B_, L_, false)
#define MX_GT_L(A_, B_)                                  \
  if (a.halves) { MX_GT_D(A_, B_, t256c::B_HALVES); }    \
  else { MX_GT_D(A_, B_, t256c::B_INTERLEAVED); }
  if (a.a_2d) {
    if (a.b_2d) { MX_GT_L(true, true) } else { MX_GT_L(true, false) }
  } else {
    if (a.b_2d) { MX_GT_L(false, true) } else { MX_GT_L(false, false) }
  }
#undef MX_GT_L
#undef MX_GT_D
#undef MX_GT
  return hipGetLastError();
}

}  // namespace mx
