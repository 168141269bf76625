// The linear layer with its epilogue on the 256x256 MXFP4 pipeline
// (gemm_tile256.h): Y = act(A B^T + bias) + residual, or the gradient dP = dY *
// act'(A B^T + bias) with the product recomputed, so that the sums of products reach
// memory in neither direction.
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

template <bool A2D, bool B2D, bool BWD>
__global__ __launch_bounds__(64 * GW, 1) void k_linear256(MxOperand A, MxOperand B, int M, int N, int K,
                                                          t256c::LinearOut lo, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[t256::LDS_BYTES];
  __shared__ t256c::LinearOut slo;
  if (threadIdx.x == 0) slo = lo;
  __syncthreads();
  const DenseSched sc{A.codes, A.scales, B.codes, B.scales, M, N, tiles_m, tiles_n,
                      XcdShare((int)blockIdx.x, (int)gridDim.x, tiles_m * tiles_n)};
  const t256::Strides sd{(int)A.ld_codes, (int)A.ld_scales, (int)B.ld_codes, (int)B.ld_scales};
  t256::run_tiles<A2D, B2D, BWD ? t256::OUT_LINEAR_BWD : t256::OUT_LINEAR, true>(sc, sd, K, nullptr, 0, lds,
                                                                                t256::QOut{}, nullptr, &slo);
}

template <bool B2D, bool BWD>
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
  t256::run_tiles<false, B2D, BWD ? t256::OUT_LINEAR_BWD : t256::OUT_LINEAR, true>(sc, sd, K, nullptr, 0, lds,
                                                                                  t256::QOut{}, nullptr, &slo);
}

}  // namespace

// The pipeline fetches scale rows 16 bytes at a time and addresses an operand,
// and a tile's rows of the buffers, with 32-bit offsets.
bool linear256_layout_ok(const GatedArgs& a) {
  const int64_t lim = 1ll << 31;
  const bool words = a.A.ld_scales % 16 == 0 && a.B.ld_scales % 16 == 0 && a.stride_scales % 16 == 0 &&
                     (uintptr_t)a.A.scales % 16 == 0 && (uintptr_t)a.B.scales % 16 == 0;
  const int64_t arows = a.offsets ? 256 : a.M;
  const bool small = arows * a.A.ld_codes < lim && a.N * a.B.ld_codes < lim && arows * a.A.ld_scales < lim &&
                     a.N * a.B.ld_scales < lim && 256 * a.ldo * 4 < lim && 256 * a.lddh * 4 < lim &&
                     a.K < (1ll << 30);
  const int64_t slots = a.offsets ? (a.M + 255) / 256 + a.E : (a.M + 255) / 256;
  return a.a_elem == 0 && a.b_elem == 0 && words && small && (!a.offsets || a.E <= GG_EMAX) &&
         slots * ((a.N + 255) / 256) < lim;
}

hipError_t launch_linear256(const GatedArgs& a, hipStream_t st) {
  const int cus = cu_count();
  const int tiles_n = (int)((a.N + 255) / 256);
  const int64_t tiles_m = a.offsets ? (a.M + 255) / 256 + a.E : (a.M + 255) / 256;
  const int64_t tiles = tiles_m * tiles_n;
  const unsigned nwg = (unsigned)(tiles < cus ? tiles : cus);
  const t256c::LinearOut lo = linear_out(a);
#define MX_LT(A_, B_, D_)                                                                                           \
  do {                                                                                                              \
    if (a.offsets) {                                                                                                \
      if constexpr (!(A_))                                                                                          \
        hipLaunchKernelGGL((k_grouped_linear256<B_, D_>), dim3(nwg), dim3(64 * GW), 0, st, a.A, a.B, a.M, (int)a.N, \
                           (int)a.K, a.offsets, a.E, a.stride_codes, a.stride_scales, lo, tiles_n);                 \
    } else {                                                                                                        \
      hipLaunchKernelGGL((k_linear256<A_, B_, D_>), dim3(nwg), dim3(64 * GW), 0, st, a.A, a.B, (int)a.M, (int)a.N,  \
                         (int)a.K, lo, (int)tiles_m, tiles_n);                                                      \
    }                                                                                                               \
  } while (0)
#define MX_LT_D(A_, B_) \
  if (a.backward) MX_LT(A_, B_, true); else MX_LT(A_, B_, false)
  if (a.a_2d) {
    if (a.b_2d) { MX_LT_D(true, true); } else { MX_LT_D(true, false); }
  } else {
    if (a.b_2d) { MX_LT_D(false, true); } else { MX_LT_D(false, false); }
  }
#undef MX_LT_D
#undef MX_LT
  return hipGetLastError();
}

}  // namespace mx
