// The linear layer with its epilogue on the 256x256 MXFP4 pipeline (gemm_tile256.h): Y =
// act(A B^T + bias) + residual, or the gradient dP = dY * act'(A B^T + bias) with the
// product recomputed, so that the sums of products reach memory in neither direction.
// One kernel per activation and direction (see the epilogue).
//
// 16384 x 2880 x 2880 with bias and residual 95-98 us (2.8 PFLOP/s; the plain product
// 72-74), SiLU 101, GELU 115, its tanh form 103, backward 102 / 115 / 106; float32
// residual and output 138.  768 tiles are three full rounds of the 256 CUs; what is over
// the plain product is the residual, whose 31 MB per round all CUs want at once, and in
// GELU its polynomial.  Experts, 65536 rows over 32, with bias 353-360 us (3.0-3.1
// PFLOP/s; the plain grouped product 346-350), 13 rounds of 272 ragged row tiles; 16384
// rows backward 147.
#pragma once

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

template <bool A2D, bool B2D, int OUT>
__global__ __launch_bounds__(64 * GW, 1) void k_linear256(MxOperand A, MxOperand B, int M, int N, int K,
                                                          t256c::LinearOut lo, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[t256::LDS_BYTES];
  __shared__ t256c::LinearOut slo;
  if (threadIdx.x == 0) slo = lo;
  __syncthreads();
  const DenseSched sc{A.codes, A.scales, B.codes, B.scales, M, N, tiles_m, tiles_n,
                      XcdShare((int)blockIdx.x, (int)gridDim.x, tiles_m * tiles_n)};
  const t256::Strides sd{(int)A.ld_codes, (int)A.ld_scales, (int)B.ld_codes, (int)B.ld_scales};
  t256::run_tiles<A2D, B2D, OUT, true>(sc, sd, K, nullptr, 0, lds, t256::QOut{}, nullptr, &slo);
}

template <bool B2D, int OUT>
__global__ __launch_bounds__(64 * GW, 1) void k_grouped_linear256(MxOperand A, MxOperand B, int64_t M_cap, int N,
                                                                  int K, const int32_t* __restrict__ offsets, int E,
                                                                  int64_t stride_codes, int64_t stride_scales,
                                                                  t256c::LinearOut lo, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[t256::LDS_BYTES];
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
  const t256::Strides sd{(int)A.ld_codes, (int)A.ld_scales, (int)B.ld_codes, (int)B.ld_scales};
  t256::run_tiles<false, B2D, OUT, true>(sc, sd, K, nullptr, 0, lds, t256::QOut{}, nullptr, &slo);
}

// OUT: an output kind of run_tiles.
template <bool A2D, bool B2D, int OUT>
hipError_t launch_out(const LinearArgs& a, hipStream_t st) {
  const int cus = cu_count();
  const int tiles_n = (int)((a.N + 255) / 256);
  const int64_t tiles_m = a.offsets ? (a.M + 255) / 256 + a.E : (a.M + 255) / 256;
  const int64_t tiles = tiles_m * tiles_n;
  const unsigned nwg = (unsigned)(tiles < cus ? tiles : cus);
  const t256c::LinearOut lo = linear_out(a);
  if constexpr (!A2D) {
    if (a.offsets) {
      hipLaunchKernelGGL((k_grouped_linear256<B2D, OUT>), dim3(nwg), dim3(64 * GW), 0, st, a.A, a.B, a.M, (int)a.N,
                         (int)a.K, a.offsets, a.E, a.stride_codes, a.stride_scales, lo, tiles_n);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((k_linear256<A2D, B2D, OUT>), dim3(nwg), dim3(64 * GW), 0, st, a.A, a.B, (int)a.M, (int)a.N,
                     (int)a.K, lo, (int)tiles_m, tiles_n);
  return hipGetLastError();
}

}  // namespace
}  // namespace mx
