// Internal launch interface between the C-ABI layer (mx_api.cpp) and the
// kernel translation units.  Arguments are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

struct QuantArgs {
  const void* src;
  int64_t R, C, ld_src;       // source [R, C], row stride in elements
  bool bf16;                  // else float32
  bool dim0;                  // blocks along dim 0 (output = quantized transpose)
  bool two_d;                 // 32x32 tiles
  bool rht;
  int sr;                     // stochastic rounding: 0 none, 1 16-bit draws, 2 8-bit draws
  uint32_t mask;
  uint64_t seed, offset;
  uint8_t* codes;
  int64_t ld_codes;
  uint8_t* scales;
  int64_t ld_scales;
  int scale_mode = 0;                // 0 reference rule, 1 round up, 2 prescale by 3/4
  const int32_t* gather = nullptr;   // device [R]: source row of each output row (last dim, 1-D only)
  int64_t R_src = 0;                 // source rows when gathering
  int elem = 0;                      // mx_elem of the output (0: FP4 E2M1)
};

struct DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, K, ld_codes, ld_scales;
  bool two_d;
  bool inverse_rht;
  uint32_t mask;
  void* dst;
  bool out_bf16;
  int64_t ld_dst;
  int elem = 0;
};

// One MX operand as the GEMM kernels see it.
struct MxOperand {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t ld_codes, ld_scales;
};

struct GemmArgs {
  MxOperand A, B;
  bool a_2d, b_2d;
  int64_t M, N, K;
  void* C;
  int64_t ldc;
  bool out_bf16;
  int a_elem = 0, b_elem = 0;  // mx_elem of A and B
};

// C = A B^T quantized along N (MXFP4, 1-D blocks, RNE) in the GEMM epilogue.
struct GemmQuantArgs {
  MxOperand A, B;
  bool a_2d, b_2d;
  int64_t M, N, K;
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld_codes, ld_scales;
  int scale_mode;
  int a_elem = 0, b_elem = 0;  // mx_elem of A and B (E2M1, or both MXFP8 / MXFP6)
};

// C = Q(A) B^T with A bf16 [M, K] (row stride lda elements) quantized to
// MXFP4 in the GEMM's operand load (RNE, 1-D blocks along K, optional
// transform with sign mask `mask`, scale_mode as mx_quantize); B MXFP4.
struct GemmQaArgs {
  const void* a;
  int64_t lda;
  bool rht;
  uint32_t mask;
  int scale_mode;
  MxOperand B;
  bool b_2d;
  int64_t M, N, K;
  void* C;
  int64_t ldc;
  bool out_bf16;
};

struct GroupedGemmArgs {
  MxOperand A, B;             // B = expert 0
  bool a_2d, b_2d;
  int64_t M_cap, N, K;
  const int32_t* offsets;     // device, E+1
  int32_t E;
  int64_t stride_codes, stride_scales;
  void* C;
  int64_t ldc;
  bool out_bf16;
  int a_elem = 0, b_elem = 0;  // mx_elem of A and B
};

// The grouped product quantized along N (MXFP4, 1-D blocks, RNE) in the
// epilogue: g describes the product (its C, ldc and out_bf16 are unused).
struct GroupedQuantArgs {
  GroupedGemmArgs g;
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld_codes, ld_scales;
  int scale_mode;
};

struct TransposeArgs {
  const uint8_t* in_codes;
  const uint8_t* in_scales;
  int64_t R, C;               // input [R, C] elements, both multiples of 32
  int64_t ld_in, ld_sin;
  uint8_t* out_codes;
  uint8_t* out_scales;
  int64_t ld_out, ld_sout;
  int bits = 4;               // bits per element code (4, 6 or 8)
};

// Compute units of the current device (cached per device).
int cu_count();

hipError_t launch_quantize(const QuantArgs& a, hipStream_t st);

// Clipping statistic: the elements that saturate when src is quantized with
// these settings, added to *count.
struct ClipArgs {
  const void* src;
  int64_t R, C, ld_src;       // source [R, C], row stride in elements
  bool bf16, dim0, two_d, rht;
  uint32_t mask;
  int scale_mode;
  int elem;
  unsigned long long* count;  // device
};
hipError_t launch_clip_count(const ClipArgs& a, hipStream_t st);
// MXFP4 RNE quantization of the a.R source rows, row t stored to output rows
// dest[t * k + j], j < k (those in [0, M)).
hipError_t launch_quantize_scatter(const QuantArgs& a, const int32_t* dest, int k, int64_t M, hipStream_t st);
hipError_t launch_transpose(const TransposeArgs& a, hipStream_t st);
hipError_t launch_dequantize(const DequantArgs& a, hipStream_t st);
hipError_t launch_gemm(const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm_qa(const GemmQaArgs& a, hipStream_t st);
// Whether the 256x256 MXFP4 pipeline takes this problem's layout (16-byte
// scale rows, operands and output under 2 GiB, M and N >= 256).
bool gemm256_layout_ok(const GemmArgs& a);
// Split-K form of the 256x256 MXFP4 GEMM (gemm_splitk.hip): the workspace it
// needs for an M x N x K problem (0 when that shape is not split), whether it
// takes this problem, and its launch (workspace of that many bytes, 256-byte
// aligned, zero-filled before its first use and left so by every launch).
size_t gemm_splitk_workspace(int64_t M, int64_t N, int64_t K);
bool gemm_splitk_applies(const GemmArgs& a);
hipError_t launch_gemm_splitk(const GemmArgs& a, void* workspace, hipStream_t st);
// The library's own split-K workspace on the current device (a static device
// array, resolved once per device): its size and its device address.
size_t gemm_splitk_scratch_bytes();
hipError_t gemm_splitk_scratch(void** ptr);
// Whether the 256x256 pipeline (the only kernel with the quantizing epilogue)
// takes this problem; launch_gemm_quantize requires it.
bool gemm_quantize_supported(const GemmQuantArgs& a);
hipError_t launch_gemm_quantize(const GemmQuantArgs& a, hipStream_t st);
hipError_t launch_grouped_gemm(const GroupedGemmArgs& a, hipStream_t st);
// Whether the 256x256 grouped pipeline (the only grouped kernel with the
// quantizing epilogue) takes this problem; launch_grouped_gemm_quantize
// requires it.
bool grouped_quantize_supported(const GroupedQuantArgs& a);
hipError_t launch_grouped_gemm_quantize(const GroupedQuantArgs& a, hipStream_t st);

// ---------------------------------------------------------------- feed-forward block
struct NormArgs {
  const void* x;
  int64_t R, C, ldx;
  bool bf16;                  // x and y (else float32)
  const void* weight;         // nullable
  const void* bias;           // nullable
  bool w_bf16;
  float eps;
  void* y;
  int64_t ldy;
  float* mean;                // nullable
  float* rstd;
};

struct NormBwdArgs {
  const void* dy;
  const void* x;
  int64_t R, C, lddy, ldx;
  bool bf16;
  const float* mean;
  const float* rstd;
  const void* weight;         // nullable
  bool w_bf16;
  void* dx;                   // nullable
  int64_t lddx;
  void* dweight;              // nullable
  void* dbias;                // nullable
  float* workspace;           // norm_backward_workspace bytes when dweight or dbias
};

struct DropoutArgs {
  const void* x;
  const void* residual;       // nullable
  void* y;
  int64_t R, C, ldx, ldr, ldy;
  bool bf16;
  uint32_t threshold;         // 0 .. 65536: dropped iff the draw is below
  uint64_t seed, offset;
};

// The gated block of an MX product (H), or with dH its projections' gradient
// (dP).  N counts hidden columns: B has 2N rows.  Dense: offsets null, rows
// [0, M).  Grouped: M is the row capacity, B expert 0.
struct GatedArgs {
  MxOperand A, B;
  bool a_2d, b_2d;
  int a_elem, b_elem;
  int64_t M, N, K;
  int act, halves;
  float alpha, limit, up_shift;   // limit +inf: no clamp
  const void* dH;             // null: forward
  int64_t lddh;
  bool dh_bf16;
  void* out;                  // H [M, N] or dP [M, 2N]
  int64_t ldo;
  bool out_bf16;
  const int32_t* offsets = nullptr;   // device, E+1
  int32_t E = 0;
  int64_t stride_codes = 0, stride_scales = 0;
};

// The linear layer (N counts the weight's rows): dH is the residual (null: none) or, with
// backward, dY; act 3 is none.  (Apart from the gated block's, whose kernels take their
// arguments as they are.)
struct LinearArgs : GatedArgs {
  bool backward = false;
  const void* bias = nullptr;         // [N], grouped [E, N] with row stride bias_stride
  bool bias_bf16 = false;
  int64_t bias_stride = 0;
};

// ---------------------------------------------------------------- expert layer
// The router (ids and weights out), or with dlogits its backward pass (ids and
// dweights in).
struct RouteArgs {
  const void* logits;
  int64_t T, ld;
  int32_t E, top;
  bool bf16;                  // logits and dlogits (else float32)
  bool sigmoid, renorm;
  float scale;
  int32_t* ids;               // [T, top]
  float* weights;             // [T, top]
  const float* dweights = nullptr;
  void* dlogits = nullptr;
  int64_t ldd = 0;
  bool vec = false;           // rows can be read a lane's logits at a time (set by the launch)
};
hipError_t launch_route(const RouteArgs& a, hipStream_t st);

struct SortArgs {
  const int32_t* ids;         // n = T * top slots
  int64_t n;
  int32_t top, E;
  int32_t* offsets;           // [E + 1]
  int32_t* rows;              // [n]
  int32_t* dest;              // [n]
  int* ws;                    // sort_workspace bytes
  int64_t chunks = 0;         // set by the launch, with the bits of an expert's number
  int bits = 0;
};
size_t sort_workspace(int64_t n, int32_t E);
hipError_t launch_expert_sort(const SortArgs& a, hipStream_t st);

// Combine, its backward pass and the dispatch (x in dout, xs in dy).
struct CombineArgs {
  int64_t T, C, rows;         // rows: of y, dy
  int32_t top;
  bool bf16;
  const int32_t* dest;        // [T, top]
  const float* weights;       // [T, top], nullable in combine
  const void* y;
  int64_t ldy;
  const void* residual;       // nullable
  int64_t ldr;
  void* out;
  int64_t ldo;
  const void* dout;
  int64_t lddo;
  void* dy;
  int64_t lddy;
  float* dweights;
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t st);
hipError_t launch_dispatch(const CombineArgs& a, hipStream_t st);
hipError_t launch_combine_backward(const CombineArgs& a, hipStream_t st);

// Column sums [E, N] of dp [M, N]: dense (offsets null, E = 1) or per expert.
struct BiasGradArgs {
  const void* dp;
  int64_t M, N, ld;
  bool bf16;
  const int32_t* offsets;     // nullable
  int32_t E;
  void* out;
  bool out_bf16;
  float* ws;                  // bias_grad_workspace bytes
};
size_t bias_grad_workspace(int64_t M, int64_t N, int32_t E, bool grouped);
bool bias_grad_fits(int64_t M, int64_t N, int32_t E, bool grouped);
hipError_t launch_bias_grad(const BiasGradArgs& a, hipStream_t st);

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t st);
size_t norm_backward_workspace(int64_t R, int64_t C);
hipError_t launch_layer_norm_backward(const NormBwdArgs& a, hipStream_t st);
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t st);
hipError_t launch_gated(const GatedArgs& a, hipStream_t st);
// The gated block on the 256x256 MXFP4 pipeline (gated256.hip): whether it
// takes this problem's types and layout, and its launch.
bool gated256_layout_ok(const GatedArgs& a);
hipError_t launch_gated256(const GatedArgs& a, hipStream_t st);
// The same on the MXFP8 / MXFP6 pipeline (gated_f8.hip).
bool gated_f8_layout_ok(const GatedArgs& a);
hipError_t launch_gated_f8(const GatedArgs& a, hipStream_t st);
// The linear layer with its epilogue, on the same kernels and pipelines.
hipError_t launch_linear(const LinearArgs& a, hipStream_t st);
bool linear256_layout_ok(const LinearArgs& a);
hipError_t launch_linear256(const LinearArgs& a, hipStream_t st);
hipError_t launch_linear256_act(const LinearArgs& a, hipStream_t st);
bool linear_f8_layout_ok(const LinearArgs& a);
hipError_t launch_linear_f8(const LinearArgs& a, hipStream_t st);
hipError_t launch_linear_f8_fp6(const LinearArgs& a, hipStream_t st);
hipError_t launch_linear_f8_backward(const LinearArgs& a, hipStream_t st);
hipError_t launch_linear_f8_backward_fp6(const LinearArgs& a, hipStream_t st);

}  // namespace mx
