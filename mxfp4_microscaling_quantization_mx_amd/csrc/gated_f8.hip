// The gated block on the direct-to-LDS pipeline for MXFP8 / MXFP6 operands
// (gemm_f8.h), any pair of E4M3, E5M2, E2M3 and E3M2: the tile order and the
// epilogues of the MXFP4 kernels.  Bound, like the plain product on it, by LDS
// reads and the operand path: 16384 x 2880 x 2880 in MXFP8 297 us, 1.83 PFLOP/s
// (the plain product with bf16 output 314), backward 340; MXFP6 295 and 342; 3000
// rows 90 for 12 x 23 tiles of 256 x 128 in two rounds on 256 CUs, 47-51 where
// one round does.
#define MX_T256_NS t256
#define MX_T256_SWAP 0
#include "gemm_tile256.h"
#undef MX_T256_NS
#undef MX_T256_SWAP
#define MX_T256_NS t256s
#define MX_T256_SWAP 1
#include "gemm_tile256.h"
#undef MX_T256_NS
#undef MX_T256_SWAP
#include "gemm_f8.h"
#include "gemm_sched.h"
#include "mx_device.h"
#include "mx_launch.h"

namespace mx {
namespace {

// (interleaved or halves is a run-time choice here)
constexpr int GATED = t256c::B_INTERLEAVED;

template <int FA, int FB>
__global__ __launch_bounds__(512, 1) void k_gated_f8(MxOperand A, MxOperand B, int M, int N, int K, t256c::GateOut go,
                                                    int halves, int a_2d, int b_2d, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t slots[2 * f8::SLOT];
  __shared__ __attribute__((aligned(16))) uint32_t sws[2 * f8::SWORDS];
  __shared__ t256c::GateOut sgo;
  if (threadIdx.x == 0) sgo = go;
  __syncthreads();
  const DenseSchedT<GATED> sc{A.codes, A.scales, B.codes, B.scales, M, N, tiles_m, tiles_n,
                              XcdShare((int)blockIdx.x, (int)gridDim.x, tiles_m * tiles_n)};
  run_f8<FA, FB, 3>(sc, A, B, K, nullptr, 0, a_2d, b_2d, slots, sws, t256::QOut{}, &sgo, halves);
}

template <int FA, int FB>
__global__ __launch_bounds__(512, 1) void k_grouped_gated_f8(MxOperand A, MxOperand B, int64_t M_cap, int N, int K,
                                                            const int32_t* __restrict__ offsets, int E,
                                                            int64_t stride_codes, int64_t stride_scales,
                                                            t256c::GateOut go, int halves, int b_2d, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t slots[2 * f8::SLOT];
  __shared__ __attribute__((aligned(16))) uint32_t sws[2 * f8::SWORDS];
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
  const GroupedSchedT<GATED> sc{&prm, tab, XcdShare((int)blockIdx.x, (int)gridDim.x, total_slots * tiles_n)};
  run_f8<FA, FB, 3>(sc, A, B, K, nullptr, 0, 0, b_2d, slots, sws, t256::QOut{}, &sgo, halves);
}

template <int FA, int FB>
hipError_t launch_f8(const GatedArgs& a, hipStream_t st) {
  const int cus = cu_count();
  const int tiles_n = (int)((a.N + 127) / 128);
  const int64_t tiles_m = a.offsets ? (a.M + 255) / 256 + a.E : (a.M + 255) / 256;
  const int64_t tiles = tiles_m * tiles_n;
  const unsigned nwg = (unsigned)(tiles < cus ? tiles : cus);
  const t256c::GateOut go{gate_params(a.act, a.alpha, a.limit, a.up_shift), a.out, a.dH, (int)a.ldo, (int)a.lddh,
                          (int)a.out_bf16, (int)a.dh_bf16};
  if (a.offsets)
    hipLaunchKernelGGL((k_grouped_gated_f8<FA, FB>), dim3(nwg), dim3(512), 0, st, a.A, a.B, a.M, (int)a.N, (int)a.K,
                       a.offsets, a.E, a.stride_codes, a.stride_scales, go, a.halves, (int)a.b_2d, tiles_n);
  else
    hipLaunchKernelGGL((k_gated_f8<FA, FB>), dim3(nwg), dim3(512), 0, st, a.A, a.B, (int)a.M, (int)a.N, (int)a.K, go,
                       a.halves, (int)a.a_2d, (int)a.b_2d, (int)tiles_m, tiles_n);
  return hipGetLastError();
}

template <int FA>
hipError_t launch_f8_b(const GatedArgs& a, hipStream_t st) {
  switch (a.b_elem) {
    case 1: return launch_f8<FA, 1>(a, st);
    case 2: return launch_f8<FA, 2>(a, st);
    case 3: return launch_f8<FA, 3>(a, st);
    default: return launch_f8<FA, 4>(a, st);
  }
}

}  // namespace

// Scale rows are fetched a 32-bit word at a time; the weight operand, 256 rows
// of A and of the buffers are addressed with 32-bit offsets.
bool gated_f8_layout_ok(const GatedArgs& a) {
  const int64_t lim = 1ll << 31;
  const bool words = a.A.ld_scales % 4 == 0 && a.B.ld_scales % 4 == 0 && a.stride_scales % 4 == 0 &&
                     (uintptr_t)a.A.scales % 4 == 0 && (uintptr_t)a.B.scales % 4 == 0;
  const bool small = 256 * a.A.ld_codes < lim && 2 * a.N * a.B.ld_codes < lim && 256 * a.A.ld_scales < lim &&
                     2 * a.N * a.B.ld_scales < lim && 256 * a.ldo * 4 < lim && 256 * a.lddh * 4 < lim &&
                     a.K < (1ll << 30);
  const int64_t slots = a.offsets ? (a.M + 255) / 256 + a.E : (a.M + 255) / 256;
  return a.a_elem >= 1 && a.b_elem >= 1 && words && small && (!a.offsets || a.E <= GG_EMAX) &&
         slots * ((a.N + 127) / 128) < lim;
}

hipError_t launch_gated_f8(const GatedArgs& a, hipStream_t st) {
  switch (a.a_elem) {
    case 1: return launch_f8_b<1>(a, st);
    case 2: return launch_f8_b<2>(a, st);
    case 3: return launch_f8_b<3>(a, st);
    default: return launch_f8_b<4>(a, st);
  }
}

}  // namespace mx
