// The linear layer with its epilogue on the direct-to-LDS pipeline for MXFP8 / MXFP6
// operands (gemm_f8.h), any pair of E4M3, E5M2, E2M3 and E3M2: the tile order and the
// epilogue of the MXFP4 kernels, the activation chosen at run time (the product is twice
// as long, and 64 kernels are enough to compile).  16384 x 2880 x 2880 with bias and
// residual: MXFP8 162 us (1.7 PFLOP/s; the plain product 150), SiLU 161, GELU 174, its tanh
// form 164, backward 166 / 174 / 167; MXFP6 153, 152, 164, 154, backward 157 / 164 / 157.
#pragma once

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

template <int FA, int FB, int OUT>
__global__ __launch_bounds__(512, 1) void k_linear_f8(MxOperand A, MxOperand B, int M, int N, int K,
                                                     t256c::LinearOut lo, int a_2d, int b_2d, int tiles_m,
                                                     int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t slots[2 * f8::SLOT];
  __shared__ __attribute__((aligned(16))) uint32_t sws[2 * f8::SWORDS];
  __shared__ t256c::LinearOut slo;
  if (threadIdx.x == 0) slo = lo;
  __syncthreads();
  const DenseSched sc{A.codes, A.scales, B.codes, B.scales, M, N, tiles_m, tiles_n,
                      XcdShare((int)blockIdx.x, (int)gridDim.x, tiles_m * tiles_n)};
  run_f8<FA, FB, OUT>(sc, A, B, K, nullptr, 0, a_2d, b_2d, slots, sws, t256::QOut{}, nullptr, 0, &slo);
}

template <int FA, int FB, int OUT>
__global__ __launch_bounds__(512, 1) void k_grouped_linear_f8(MxOperand A, MxOperand B, int64_t M_cap, int N, int K,
                                                             const int32_t* __restrict__ offsets, int E,
                                                             int64_t stride_codes, int64_t stride_scales,
                                                             t256c::LinearOut lo, int b_2d, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t slots[2 * f8::SLOT];
  __shared__ __attribute__((aligned(16))) uint32_t sws[2 * f8::SWORDS];
  __shared__ int tab[3 * GG_EMAX + 1];
  __shared__ GroupedParams prm;
  __shared__ t256c::LinearOut slo;
  build_expert_table(offsets, E, M_cap, tab);   // ends with a barrier
  const int total_slots = tab[E];
  if (threadIdx.x == 0) {
    prm = GroupedParams{A.codes, A.scales, B.codes, B.scales, stride_codes, stride_scales, (int)A.ld_codes,
                        (int)A.ld_scales, N, tiles_n, E, total_slots, 0, 0};
    slo = lo;
  }
  __syncthreads();
  const GroupedSched sc{&prm, tab, XcdShare((int)blockIdx.x, (int)gridDim.x, total_slots * tiles_n)};
  run_f8<FA, FB, OUT>(sc, A, B, K, nullptr, 0, 0, b_2d, slots, sws, t256::QOut{}, nullptr, 0, &slo);
}

template <int FA, int FB, int OUT>
hipError_t launch_f8(const LinearArgs& a, hipStream_t st) {
  const int cus = cu_count();
  const int tiles_n = (int)((a.N + 255) / 256);
  const int64_t tiles_m = a.offsets ? (a.M + 255) / 256 + a.E : (a.M + 255) / 256;
  const int64_t tiles = tiles_m * tiles_n;
  const unsigned nwg = (unsigned)(tiles < cus ? tiles : cus);
  const t256c::LinearOut lo = linear_out(a);
  if (a.offsets)
    hipLaunchKernelGGL((k_grouped_linear_f8<FA, FB, OUT>), dim3(nwg), dim3(512), 0, st, a.A, a.B, a.M, (int)a.N,
                       (int)a.K, a.offsets, a.E, a.stride_codes, a.stride_scales, lo, (int)a.b_2d, tiles_n);
  else
    hipLaunchKernelGGL((k_linear_f8<FA, FB, OUT>), dim3(nwg), dim3(512), 0, st, a.A, a.B, (int)a.M, (int)a.N,
                       (int)a.K, lo, (int)a.a_2d, (int)a.b_2d, (int)tiles_m, tiles_n);
  return hipGetLastError();
}

template <int FA, int OUT>
hipError_t launch_f8_b(const LinearArgs& a, hipStream_t st) {
  switch (a.b_elem) {
    case 1: return launch_f8<FA, 1, OUT>(a, st);
    case 2: return launch_f8<FA, 2, OUT>(a, st);
    case 3: return launch_f8<FA, 3, OUT>(a, st);
    default: return launch_f8<FA, 4, OUT>(a, st);
  }
}

}  // namespace

}  // namespace mx
