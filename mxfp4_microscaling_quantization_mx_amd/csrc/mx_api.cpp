// C-ABI entry points of libmxfp4: argument validation, error reporting and
// dispatch to the kernel launchers.  Declarations and the contract of every
// entry point are in include/mx.h.
#include "../../include/mx.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "mx_launch.h"

namespace {

thread_local char g_err[512] = "";

mx_status fail(mx_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

mx_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return MX_OK;
  return fail(MX_ERR_HIP, "%s: HIP error %d (%s)", what, (int)e, hipGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Validate one MX operand description; `what` names it in messages.
// Bits per element of an mx_elem (0 for an unknown value).
int elem_bits(int32_t e) {
  switch (e) {
    case MX_ELEM_E2M1: return 4;
    case MX_ELEM_E4M3:
    case MX_ELEM_E5M2: return 8;
    case MX_ELEM_E2M3:
    case MX_ELEM_E3M2: return 6;
    default: return 0;
  }
}

mx_status check_tensor(const mx_tensor* t, const char* what) {
  if (!t) return fail(MX_ERR_INVALID_ARG, "%s: null mx_tensor", what);
  if (t->rows < 0 || t->K < 0) return fail(MX_ERR_INVALID_ARG, "%s: negative shape", what);
  if (t->K % 32) return fail(MX_ERR_INVALID_ARG, "%s: K=%lld is not a multiple of 32", what, (long long)t->K);
  if (t->block != MX_BLOCK_1D && t->block != MX_BLOCK_2D)
    return fail(MX_ERR_INVALID_ARG, "%s: unknown block kind %d", what, t->block);
  if (elem_bits(t->elem) == 0) return fail(MX_ERR_INVALID_ARG, "%s: unknown element type %d", what, t->elem);
  if (t->block == MX_BLOCK_2D && t->rows % 32)
    return fail(MX_ERR_INVALID_ARG, "%s: 2-D blocks need rows %% 32 == 0 (rows=%lld)", what, (long long)t->rows);
  if (t->rows == 0 || t->K == 0) return MX_OK;
  if (!t->codes || !t->scales) return fail(MX_ERR_INVALID_ARG, "%s: null codes/scales pointer", what);
  if (t->ld_codes < t->K * elem_bits(t->elem) / 8 || t->ld_scales < t->K / 32)
    return fail(MX_ERR_INVALID_ARG, "%s: row strides too small (ld_codes=%lld, ld_scales=%lld)", what,
                (long long)t->ld_codes, (long long)t->ld_scales);
  if (!aligned(t->codes, 16) || t->ld_codes % 16)
    return fail(MX_ERR_INVALID_ARG, "%s: codes must be 16-byte aligned with ld_codes %% 16 == 0", what);
  return MX_OK;
}

mx::MxOperand operand(const mx_tensor* t) {
  return mx::MxOperand{t->codes, t->scales, t->ld_codes, t->ld_scales};
}

// The C++ kernels for MXFP8 / MXFP6 operands (and the operand-load
// quantizing GEMM) address one 256-row tile of an operand, of its scales and
// of C with 32-bit buffer offsets.
bool tile_offsets_fit(const mx_tensor* t, int64_t ldc_bytes) {
  const int64_t lim = (int64_t)1 << 31;
  return (t == nullptr || (256 * t->ld_codes < lim && 256 * t->ld_scales < lim)) && 256 * ldc_bytes < lim;
}

}  // namespace

extern "C" {

const char* mx_last_error(void) { return g_err; }

const char* mx_version(void) { return "libmxfp4 0.1.0 (gfx950)"; }

mx_status mx_quantize(const void* src, int32_t src_dtype, int64_t R, int64_t C, int64_t ld_src,
                      const mx_quant_cfg* cfg, const mx_tensor* out, void* stream) {
  g_err[0] = '\0';
  if (!cfg || !out) return fail(MX_ERR_INVALID_ARG, "mx_quantize: null cfg or out");
  if (src_dtype != MX_DT_F32 && src_dtype != MX_DT_BF16)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize: unknown source dtype %d", src_dtype);
  if (cfg->axis != MX_AXIS_LAST && cfg->axis != MX_AXIS_DIM0)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize: unknown axis %d", cfg->axis);
  if (cfg->rounding != MX_ROUND_RNE && cfg->rounding != MX_ROUND_SR && cfg->rounding != MX_ROUND_SR8)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize: unknown rounding %d", cfg->rounding);
  if (cfg->block != MX_BLOCK_1D && cfg->block != MX_BLOCK_2D)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize: unknown block kind %d", cfg->block);
  if (cfg->use_rht != 0 && cfg->use_rht != 1)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize: use_rht must be 0 or 1");
  if (cfg->scale_mode > MX_SCALE_PRESCALE_3_4)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize: unknown scale_mode %u", cfg->scale_mode);
  if (R < 0 || C < 0) return fail(MX_ERR_INVALID_ARG, "mx_quantize: negative shape");
  const bool dim0 = cfg->axis == MX_AXIS_DIM0;
  const int64_t rows_out = dim0 ? C : R;
  const int64_t K = dim0 ? R : C;
  if (K % 32) return fail(MX_ERR_INVALID_ARG, "mx_quantize: blocking dimension %lld is not a multiple of 32", (long long)K);
  if (out->rows != rows_out || out->K != K)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize: out is [%lld, %lld], expected [%lld, %lld]",
                (long long)out->rows, (long long)out->K, (long long)rows_out, (long long)K);
  if (out->block != cfg->block) return fail(MX_ERR_INVALID_ARG, "mx_quantize: out->block differs from cfg->block");
  mx_status st = check_tensor(out, "mx_quantize: out");
  if (st != MX_OK) return st;
  if (R == 0 || C == 0) return MX_OK;
  if (!src) return fail(MX_ERR_INVALID_ARG, "mx_quantize: null src");
  if (ld_src < C) return fail(MX_ERR_INVALID_ARG, "mx_quantize: ld_src=%lld < C=%lld", (long long)ld_src, (long long)C);
  // along the last dim the kernels read 16-byte pieces of a row; along dim 0
  // one element per lane, so any element-aligned base and row stride will do
  if (dim0 ? !aligned(src, src_dtype == MX_DT_BF16 ? 2 : 4) : (!aligned(src, 16) || ld_src % 8))
    return fail(MX_ERR_INVALID_ARG,
                dim0 ? "mx_quantize: src must be aligned to its element size"
                     : "mx_quantize: src must be 16-byte aligned with ld_src %% 8 == 0 (blocks along the last dim)");
  if (dim0 && (R + 127) / 128 > 65535)
    return fail(MX_ERR_UNSUPPORTED, "mx_quantize: dim-0 blocking supports at most 65535*128 source rows");
  if (dim0 && (31 * ld_src + C) * (src_dtype == MX_DT_BF16 ? 2 : 4) > (int64_t)0xFFFFFFFF)
    return fail(MX_ERR_UNSUPPORTED, "mx_quantize: dim-0 blocking needs 32 source rows to span < 4 GiB");
  if (!dim0 && R * (C / 32) > (int64_t)0xFFFFFF00)
    return fail(MX_ERR_UNSUPPORTED, "mx_quantize: at most 2^32 - 256 blocks per call");

  mx::QuantArgs a{};
  a.src = src;
  a.R = R;
  a.C = C;
  a.ld_src = ld_src;
  a.bf16 = src_dtype == MX_DT_BF16;
  a.dim0 = dim0;
  a.two_d = cfg->block == MX_BLOCK_2D;
  a.rht = cfg->use_rht == 1;
  a.sr = cfg->rounding == MX_ROUND_SR ? 1 : cfg->rounding == MX_ROUND_SR8 ? 2 : 0;
  a.mask = cfg->rht_sign_mask;
  a.seed = cfg->philox_seed;
  a.offset = cfg->philox_offset;
  a.scale_mode = (int)cfg->scale_mode;
  a.codes = out->codes;
  a.ld_codes = out->ld_codes;
  a.scales = out->scales;
  a.ld_scales = out->ld_scales;
  a.elem = out->elem;
  return hip_status(mx::launch_quantize(a, static_cast<hipStream_t>(stream)), "mx_quantize");
}

mx_status mx_clip_count(const void* src, int32_t src_dtype, int64_t R, int64_t C, int64_t ld_src,
                        const mx_quant_cfg* cfg, int32_t elem, uint64_t* count, void* stream) {
  g_err[0] = '\0';
  if (!cfg) return fail(MX_ERR_INVALID_ARG, "mx_clip_count: null cfg");
  if (src_dtype != MX_DT_F32 && src_dtype != MX_DT_BF16)
    return fail(MX_ERR_INVALID_ARG, "mx_clip_count: unknown source dtype %d", src_dtype);
  if (cfg->axis != MX_AXIS_LAST && cfg->axis != MX_AXIS_DIM0)
    return fail(MX_ERR_INVALID_ARG, "mx_clip_count: unknown axis %d", cfg->axis);
  if (cfg->block != MX_BLOCK_1D && cfg->block != MX_BLOCK_2D)
    return fail(MX_ERR_INVALID_ARG, "mx_clip_count: unknown block kind %d", cfg->block);
  if (cfg->use_rht != 0 && cfg->use_rht != 1)
    return fail(MX_ERR_INVALID_ARG, "mx_clip_count: use_rht must be 0 or 1");
  if (cfg->scale_mode > MX_SCALE_PRESCALE_3_4)
    return fail(MX_ERR_INVALID_ARG, "mx_clip_count: unknown scale_mode %u", cfg->scale_mode);
  if (elem < MX_ELEM_E2M1 || elem > MX_ELEM_E3M2)
    return fail(MX_ERR_INVALID_ARG, "mx_clip_count: unknown element type %d", elem);
  if (R < 0 || C < 0) return fail(MX_ERR_INVALID_ARG, "mx_clip_count: negative shape");
  const bool dim0 = cfg->axis == MX_AXIS_DIM0;
  const int64_t rows_out = dim0 ? C : R;
  const int64_t K = dim0 ? R : C;
  if (K % 32) return fail(MX_ERR_INVALID_ARG, "mx_clip_count: blocking dimension %lld is not a multiple of 32", (long long)K);
  if (cfg->block == MX_BLOCK_2D && rows_out % 32)
    return fail(MX_ERR_INVALID_ARG, "mx_clip_count: 2-D blocks need rows_out %% 32 == 0 (got %lld)", (long long)rows_out);
  if (!count) return fail(MX_ERR_INVALID_ARG, "mx_clip_count: null count");
  if (!aligned(count, 8)) return fail(MX_ERR_INVALID_ARG, "mx_clip_count: count must be 8-byte aligned");
  if (R == 0 || C == 0) return MX_OK;
  if (!src) return fail(MX_ERR_INVALID_ARG, "mx_clip_count: null src");
  if (ld_src < C) return fail(MX_ERR_INVALID_ARG, "mx_clip_count: ld_src=%lld < C=%lld", (long long)ld_src, (long long)C);
  // (along dim 0 the kernel reads one element per lane, as the quantizer does)
  if (dim0 ? !aligned(src, src_dtype == MX_DT_BF16 ? 2 : 4) : (!aligned(src, 16) || ld_src % 8))
    return fail(MX_ERR_INVALID_ARG,
                dim0 ? "mx_clip_count: src must be aligned to its element size"
                     : "mx_clip_count: src must be 16-byte aligned with ld_src %% 8 == 0 (blocks along the last dim)");
  mx::ClipArgs a{};
  a.src = src;
  a.R = R;
  a.C = C;
  a.ld_src = ld_src;
  a.bf16 = src_dtype == MX_DT_BF16;
  a.dim0 = dim0;
  a.two_d = cfg->block == MX_BLOCK_2D;
  a.rht = cfg->use_rht == 1;
  a.mask = cfg->rht_sign_mask;
  a.scale_mode = (int)cfg->scale_mode;
  a.elem = elem;
  a.count = reinterpret_cast<unsigned long long*>(count);
  return hip_status(mx::launch_clip_count(a, static_cast<hipStream_t>(stream)), "mx_clip_count");
}

mx_status mx_quantize_scatter(const void* src, int32_t src_dtype, int64_t R, int64_t C, int64_t ld_src,
                              const int32_t* dest, int32_t k, const mx_quant_cfg* cfg, const mx_tensor* out,
                              void* stream) {
  g_err[0] = '\0';
  if (!cfg || !out) return fail(MX_ERR_INVALID_ARG, "mx_quantize_scatter: null cfg or out");
  if (src_dtype != MX_DT_F32 && src_dtype != MX_DT_BF16)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize_scatter: unknown source dtype %d", src_dtype);
  if (cfg->axis != MX_AXIS_LAST || cfg->block != MX_BLOCK_1D)
    return fail(MX_ERR_UNSUPPORTED, "mx_quantize_scatter: only 1-D blocks along the last dim");
  if (cfg->rounding != MX_ROUND_RNE)
    return fail(MX_ERR_UNSUPPORTED, "mx_quantize_scatter: RNE only (SR draws depend on the destination row)");
  if (cfg->use_rht != 0 && cfg->use_rht != 1)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize_scatter: use_rht must be 0 or 1");
  if (cfg->scale_mode > MX_SCALE_PRESCALE_3_4)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize_scatter: unknown scale_mode %u", cfg->scale_mode);
  if (R < 0 || C < 0 || k < 0) return fail(MX_ERR_INVALID_ARG, "mx_quantize_scatter: negative shape or k");
  if (C % 32) return fail(MX_ERR_INVALID_ARG, "mx_quantize_scatter: C=%lld is not a multiple of 32", (long long)C);
  if (out->K != C)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize_scatter: out.K=%lld != C=%lld", (long long)out->K, (long long)C);
  if (out->block != MX_BLOCK_1D) return fail(MX_ERR_INVALID_ARG, "mx_quantize_scatter: out must hold 1-D blocks");
  mx_status st = check_tensor(out, "mx_quantize_scatter: out");
  if (st != MX_OK) return st;
  if (out->elem != MX_ELEM_E2M1) return fail(MX_ERR_UNSUPPORTED, "mx_quantize_scatter: MXFP4 output only");
  if (R == 0 || C == 0 || k == 0 || out->rows == 0) return MX_OK;
  if (!dest || !aligned(dest, 4)) return fail(MX_ERR_INVALID_ARG, "mx_quantize_scatter: null or unaligned dest");
  if (!src) return fail(MX_ERR_INVALID_ARG, "mx_quantize_scatter: null src");
  if (ld_src < C)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize_scatter: ld_src=%lld < C=%lld", (long long)ld_src, (long long)C);
  if (!aligned(src, 16) || ld_src % 8)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize_scatter: src must be 16-byte aligned with ld_src %% 8 == 0");
  if (R * (C / 32) > (int64_t)0xFFFFFF00)
    return fail(MX_ERR_UNSUPPORTED, "mx_quantize_scatter: at most 2^32 - 256 blocks per call");
  mx::QuantArgs a{};
  a.src = src;
  a.R = R;
  a.C = C;
  a.ld_src = ld_src;
  a.bf16 = src_dtype == MX_DT_BF16;
  a.rht = cfg->use_rht == 1;
  a.mask = cfg->rht_sign_mask;
  a.scale_mode = (int)cfg->scale_mode;
  a.codes = out->codes;
  a.ld_codes = out->ld_codes;
  a.scales = out->scales;
  a.ld_scales = out->ld_scales;
  return hip_status(mx::launch_quantize_scatter(a, dest, k, out->rows, static_cast<hipStream_t>(stream)),
                    "mx_quantize_scatter");
}

mx_status mx_quantize_gather(const void* src, int32_t src_dtype, int64_t R_src, int64_t C, int64_t ld_src,
                             const int32_t* rows, int64_t rows_out, const mx_quant_cfg* cfg,
                             const mx_tensor* out, void* stream) {
  g_err[0] = '\0';
  if (!cfg || !out) return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: null cfg or out");
  if (src_dtype != MX_DT_F32 && src_dtype != MX_DT_BF16)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: unknown source dtype %d", src_dtype);
  if (cfg->axis != MX_AXIS_LAST || cfg->block != MX_BLOCK_1D)
    return fail(MX_ERR_UNSUPPORTED, "mx_quantize_gather: only 1-D blocks along the last dim");
  if (cfg->rounding != MX_ROUND_RNE && cfg->rounding != MX_ROUND_SR && cfg->rounding != MX_ROUND_SR8)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: unknown rounding %d", cfg->rounding);
  if (cfg->use_rht != 0 && cfg->use_rht != 1)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: use_rht must be 0 or 1");
  if (cfg->scale_mode > MX_SCALE_PRESCALE_3_4)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: unknown scale_mode %u", cfg->scale_mode);
  if (R_src < 0 || C < 0 || rows_out < 0) return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: negative shape");
  if (C % 32) return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: C=%lld is not a multiple of 32", (long long)C);
  if (out->rows != rows_out || out->K != C)
    return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: out is [%lld, %lld], expected [%lld, %lld]",
                (long long)out->rows, (long long)out->K, (long long)rows_out, (long long)C);
  if (out->block != MX_BLOCK_1D) return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: out must hold 1-D blocks");
  mx_status st = check_tensor(out, "mx_quantize_gather: out");
  if (st != MX_OK) return st;
  if (out->elem != MX_ELEM_E2M1) return fail(MX_ERR_UNSUPPORTED, "mx_quantize_gather: MXFP4 output only");
  if (rows_out == 0 || C == 0) return MX_OK;
  if (!rows || !aligned(rows, 4)) return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: null or unaligned rows");
  if (R_src > 0) {
    if (!src) return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: null src");
    if (ld_src < C)
      return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: ld_src=%lld < C=%lld", (long long)ld_src, (long long)C);
    if (!aligned(src, 16) || ld_src % 8)
      return fail(MX_ERR_INVALID_ARG, "mx_quantize_gather: src must be 16-byte aligned with ld_src %% 8 == 0");
  }
  if (rows_out * (C / 32) > (int64_t)0xFFFFFF00)
    return fail(MX_ERR_UNSUPPORTED, "mx_quantize_gather: at most 2^32 - 256 blocks per call");

  mx::QuantArgs a{};
  a.src = src;
  a.R = rows_out;
  a.C = C;
  a.ld_src = ld_src;
  a.bf16 = src_dtype == MX_DT_BF16;
  a.rht = cfg->use_rht == 1;
  a.sr = cfg->rounding == MX_ROUND_SR ? 1 : cfg->rounding == MX_ROUND_SR8 ? 2 : 0;
  a.mask = cfg->rht_sign_mask;
  a.seed = cfg->philox_seed;
  a.offset = cfg->philox_offset;
  a.scale_mode = (int)cfg->scale_mode;
  a.codes = out->codes;
  a.ld_codes = out->ld_codes;
  a.scales = out->scales;
  a.ld_scales = out->ld_scales;
  a.gather = rows;
  a.R_src = R_src;
  return hip_status(mx::launch_quantize(a, static_cast<hipStream_t>(stream)), "mx_quantize_gather");
}

mx_status mx_dequantize(const mx_tensor* in, int32_t inverse_rht, uint32_t rht_sign_mask, void* dst,
                        int32_t dst_dtype, int64_t ld_dst, void* stream) {
  g_err[0] = '\0';
  mx_status st = check_tensor(in, "mx_dequantize: in");
  if (st != MX_OK) return st;
  if (dst_dtype != MX_DT_F32 && dst_dtype != MX_DT_BF16)
    return fail(MX_ERR_INVALID_ARG, "mx_dequantize: unknown destination dtype %d", dst_dtype);
  if (inverse_rht != 0 && inverse_rht != 1)
    return fail(MX_ERR_INVALID_ARG, "mx_dequantize: inverse_rht must be 0 or 1");
  if (in->rows == 0 || in->K == 0) return MX_OK;
  if (!dst) return fail(MX_ERR_INVALID_ARG, "mx_dequantize: null dst");
  if (ld_dst < in->K || ld_dst % 8 || !aligned(dst, 16))
    return fail(MX_ERR_INVALID_ARG, "mx_dequantize: dst must be 16-byte aligned with ld_dst >= K and ld_dst %% 8 == 0");
  mx::DequantArgs a{};
  a.codes = in->codes;
  a.scales = in->scales;
  a.rows = in->rows;
  a.K = in->K;
  a.ld_codes = in->ld_codes;
  a.ld_scales = in->ld_scales;
  a.two_d = in->block == MX_BLOCK_2D;
  a.inverse_rht = inverse_rht == 1;
  a.mask = rht_sign_mask;
  a.dst = dst;
  a.out_bf16 = dst_dtype == MX_DT_BF16;
  a.ld_dst = ld_dst;
  a.elem = in->elem;
  return hip_status(mx::launch_dequantize(a, static_cast<hipStream_t>(stream)), "mx_dequantize");
}

mx_status mx_transpose(const mx_tensor* in, const mx_tensor* out, void* stream) {
  g_err[0] = '\0';
  mx_status st = check_tensor(in, "mx_transpose: in");
  if (st != MX_OK) return st;
  st = check_tensor(out, "mx_transpose: out");
  if (st != MX_OK) return st;
  if (in->block != MX_BLOCK_2D || out->block != MX_BLOCK_2D)
    return fail(MX_ERR_UNSUPPORTED, "mx_transpose: only operands with 2-D (32x32) blocks transpose exactly");
  if (in->elem != out->elem)
    return fail(MX_ERR_INVALID_ARG, "mx_transpose: in and out element types differ");
  if (out->rows != in->K || out->K != in->rows)
    return fail(MX_ERR_INVALID_ARG, "mx_transpose: out is [%lld, %lld], expected [%lld, %lld]", (long long)out->rows,
                (long long)out->K, (long long)in->K, (long long)in->rows);
  if (in->rows == 0 || in->K == 0) return MX_OK;
  if (((in->rows + 127) / 128) * ((in->K + 127) / 128) > (int64_t)0x7FFFFFFF)
    return fail(MX_ERR_UNSUPPORTED, "mx_transpose: at most 2^31 - 1 tiles of 128 x 128");
  mx::TransposeArgs a{};
  a.in_codes = in->codes;
  a.in_scales = in->scales;
  a.R = in->rows;
  a.C = in->K;
  a.ld_in = in->ld_codes;
  a.ld_sin = in->ld_scales;
  a.out_codes = out->codes;
  a.out_scales = out->scales;
  a.ld_out = out->ld_codes;
  a.ld_sout = out->ld_scales;
  a.bits = elem_bits(in->elem);
  return hip_status(mx::launch_transpose(a, static_cast<hipStream_t>(stream)), "mx_transpose");
}

size_t mx_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  return mx::gemm_splitk_workspace(M, N, K);
}

namespace {

// Validate an mx_gemm call and describe it; M = 0 or N = 0 leaves a.M or a.N 0.
mx_status gemm_args(const mx_tensor* A, const mx_tensor* B, void* C, int32_t c_dtype, int64_t ldc,
                    const char* what, mx::GemmArgs& a) {
  char name[64];
  std::snprintf(name, sizeof(name), "%s: A", what);
  mx_status st = check_tensor(A, name);
  if (st != MX_OK) return st;
  std::snprintf(name, sizeof(name), "%s: B", what);
  st = check_tensor(B, name);
  if (st != MX_OK) return st;
  if (A->K != B->K)
    return fail(MX_ERR_INVALID_ARG, "%s: A.K=%lld != B.K=%lld", what, (long long)A->K, (long long)B->K);
  if (c_dtype != MX_DT_F32 && c_dtype != MX_DT_BF16)
    return fail(MX_ERR_INVALID_ARG, "%s: unknown output dtype %d", what, c_dtype);
  const int64_t M = A->rows, N = B->rows;
  a = mx::GemmArgs{};
  a.M = M;
  a.N = N;
  if (M == 0 || N == 0) return MX_OK;
  if (!C) return fail(MX_ERR_INVALID_ARG, "%s: null C", what);
  if (ldc < N) return fail(MX_ERR_INVALID_ARG, "%s: ldc=%lld < N=%lld", what, (long long)ldc, (long long)N);
  if ((M + 127) / 128 > 65535) return fail(MX_ERR_UNSUPPORTED, "%s: M too large", what);
  a.A = operand(A);
  a.B = operand(B);
  a.a_2d = A->block == MX_BLOCK_2D;
  a.b_2d = B->block == MX_BLOCK_2D;
  a.K = A->K;
  a.C = C;
  a.ldc = ldc;
  a.out_bf16 = c_dtype == MX_DT_BF16;
  a.a_elem = A->elem;
  a.b_elem = B->elem;
  if ((a.a_elem != 0 || a.b_elem != 0) &&
      !(tile_offsets_fit(A, ldc * (a.out_bf16 ? 2 : 4)) && tile_offsets_fit(B, 0)))
    return fail(MX_ERR_UNSUPPORTED, "%s: row strides too large for the MXFP8/MXFP6 kernels", what);
  return MX_OK;
}

}  // namespace

mx_status mx_gemm(const mx_tensor* A, const mx_tensor* B, void* C, int32_t c_dtype, int64_t ldc,
                  void* workspace, size_t ws_bytes, void* stream) {
  g_err[0] = '\0';
  mx::GemmArgs a;
  const mx_status st = gemm_args(A, B, C, c_dtype, ldc, "mx_gemm", a);
  if (st != MX_OK || a.M == 0 || a.N == 0) return st;
  if (a.K > 0 && mx::gemm_splitk_applies(a)) {
    const size_t need = mx::gemm_splitk_workspace(a.M, a.N, a.K);
    if (!workspace || ws_bytes < need || !aligned(workspace, 256))
      return fail(MX_ERR_INVALID_ARG,
                  "mx_gemm: this shape is split along K and needs a 256-byte aligned workspace of %zu bytes "
                  "(got %zu bytes at %p)",
                  need, ws_bytes, workspace);
    return hip_status(mx::launch_gemm_splitk(a, workspace, static_cast<hipStream_t>(stream)), "mx_gemm");
  }
  return hip_status(mx::launch_gemm(a, static_cast<hipStream_t>(stream)), "mx_gemm");
}

mx_status mx_gemm_noalloc(const mx_tensor* A, const mx_tensor* B, void* C, int32_t c_dtype, int64_t ldc,
                          void* stream) {
  g_err[0] = '\0';
  mx::GemmArgs a;
  const mx_status st = gemm_args(A, B, C, c_dtype, ldc, "mx_gemm_noalloc", a);
  if (st != MX_OK || a.M == 0 || a.N == 0) return st;
  if (a.K > 0 && mx::gemm_splitk_applies(a)) {
    const size_t need = mx::gemm_splitk_workspace(a.M, a.N, a.K);
    if (need > mx::gemm_splitk_scratch_bytes())
      return fail(MX_ERR_UNSUPPORTED,
                  "mx_gemm_noalloc: this shape's split-K workspace (%zu bytes) exceeds the library's scratch "
                  "(%zu bytes); use mx_gemm with a workspace",
                  need, mx::gemm_splitk_scratch_bytes());
    void* scratch = nullptr;
    const hipError_t e = mx::gemm_splitk_scratch(&scratch);
    if (e != hipSuccess) return hip_status(e, "mx_gemm_noalloc: scratch address");
    return hip_status(mx::launch_gemm_splitk(a, scratch, static_cast<hipStream_t>(stream)), "mx_gemm_noalloc");
  }
  return hip_status(mx::launch_gemm(a, static_cast<hipStream_t>(stream)), "mx_gemm_noalloc");
}

mx_status mx_gemm_fused_quant_a(const void* a, int32_t a_dtype, int64_t M, int64_t K, int64_t lda,
                                const mx_quant_cfg* cfg, const mx_tensor* B, void* C, int32_t c_dtype, int64_t ldc,
                                void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_gemm_fused_quant_a";
  if (!cfg || !B) return fail(MX_ERR_INVALID_ARG, "%s: null cfg or B", what);
  if (a_dtype != MX_DT_F32 && a_dtype != MX_DT_BF16)
    return fail(MX_ERR_INVALID_ARG, "%s: unknown A dtype %d", what, a_dtype);
  if (a_dtype != MX_DT_BF16) return fail(MX_ERR_UNSUPPORTED, "%s: A must be bf16", what);
  if (cfg->axis != MX_AXIS_LAST || cfg->block != MX_BLOCK_1D || cfg->rounding != MX_ROUND_RNE)
    return fail(MX_ERR_UNSUPPORTED, "%s: A is quantized along K with 1-D blocks and RNE only", what);
  if (cfg->use_rht != 0 && cfg->use_rht != 1) return fail(MX_ERR_INVALID_ARG, "%s: use_rht must be 0 or 1", what);
  if (cfg->scale_mode > MX_SCALE_PRESCALE_3_4)
    return fail(MX_ERR_INVALID_ARG, "%s: unknown scale_mode %u", what, cfg->scale_mode);
  mx_status st = check_tensor(B, "mx_gemm_fused_quant_a: B");
  if (st != MX_OK) return st;
  if (B->elem != MX_ELEM_E2M1) return fail(MX_ERR_UNSUPPORTED, "%s: B must be MXFP4", what);
  if (M < 0 || K < 0) return fail(MX_ERR_INVALID_ARG, "%s: negative shape", what);
  if (K % 32) return fail(MX_ERR_INVALID_ARG, "%s: K=%lld is not a multiple of 32", what, (long long)K);
  if (B->K != K) return fail(MX_ERR_INVALID_ARG, "%s: K=%lld != B.K=%lld", what, (long long)K, (long long)B->K);
  if (c_dtype != MX_DT_F32 && c_dtype != MX_DT_BF16)
    return fail(MX_ERR_INVALID_ARG, "%s: unknown output dtype %d", what, c_dtype);
  const int64_t N = B->rows;
  if (M == 0 || N == 0) return MX_OK;
  if (!C) return fail(MX_ERR_INVALID_ARG, "%s: null C", what);
  if (ldc < N) return fail(MX_ERR_INVALID_ARG, "%s: ldc=%lld < N=%lld", what, (long long)ldc, (long long)N);
  if (K > 0) {
    if (!a) return fail(MX_ERR_INVALID_ARG, "%s: null A", what);
    if (lda < K) return fail(MX_ERR_INVALID_ARG, "%s: lda=%lld < K=%lld", what, (long long)lda, (long long)K);
    if (!aligned(a, 16) || lda % 8)
      return fail(MX_ERR_INVALID_ARG, "%s: A must be 16-byte aligned with lda %% 8 == 0", what);
  }
  if ((M + 255) / 256 > 65535) return fail(MX_ERR_UNSUPPORTED, "%s: M too large", what);
  if (256 * lda * 2 >= ((int64_t)1 << 31) || !tile_offsets_fit(B, ldc * (c_dtype == MX_DT_BF16 ? 2 : 4)))
    return fail(MX_ERR_UNSUPPORTED, "%s: row strides too large", what);
  mx::GemmQaArgs q{};
  q.a = a;
  q.lda = lda;
  q.rht = cfg->use_rht == 1;
  q.mask = cfg->rht_sign_mask;
  q.scale_mode = (int)cfg->scale_mode;
  q.B = operand(B);
  q.b_2d = B->block == MX_BLOCK_2D;
  q.M = M;
  q.N = N;
  q.K = K;
  q.C = C;
  q.ldc = ldc;
  q.out_bf16 = c_dtype == MX_DT_BF16;
  return hip_status(mx::launch_gemm_qa(q, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_gemm_quantize(const mx_tensor* A, const mx_tensor* B, int32_t scale_mode, mx_tensor* out,
                           void* stream) {
  g_err[0] = '\0';
  mx_status st = check_tensor(A, "mx_gemm_quantize: A");
  if (st != MX_OK) return st;
  st = check_tensor(B, "mx_gemm_quantize: B");
  if (st != MX_OK) return st;
  st = check_tensor(out, "mx_gemm_quantize: out");
  if (st != MX_OK) return st;
  if (A->K != B->K)
    return fail(MX_ERR_INVALID_ARG, "mx_gemm_quantize: A.K=%lld != B.K=%lld", (long long)A->K, (long long)B->K);
  if (scale_mode < MX_SCALE_FLOOR || scale_mode > MX_SCALE_PRESCALE_3_4)
    return fail(MX_ERR_INVALID_ARG, "mx_gemm_quantize: unknown scale mode %d", scale_mode);
  const int64_t M = A->rows, N = B->rows;
  if (out->rows != M || out->K != N)
    return fail(MX_ERR_INVALID_ARG, "mx_gemm_quantize: out is [%lld, %lld], the product is [%lld, %lld]",
                (long long)out->rows, (long long)out->K, (long long)M, (long long)N);
  if (out->elem != MX_ELEM_E2M1) return fail(MX_ERR_UNSUPPORTED, "mx_gemm_quantize: the output is MXFP4");
  if ((A->elem == MX_ELEM_E2M1) != (B->elem == MX_ELEM_E2M1))
    return fail(MX_ERR_UNSUPPORTED, "mx_gemm_quantize: both operands MXFP4, or both MXFP8 / MXFP6");
  if (out->block != MX_BLOCK_1D)
    return fail(MX_ERR_UNSUPPORTED, "mx_gemm_quantize: the output uses 1-D blocks");
  if (M == 0 || N == 0) return MX_OK;
  mx::GemmQuantArgs a{};
  a.A = operand(A);
  a.B = operand(B);
  a.a_2d = A->block == MX_BLOCK_2D;
  a.b_2d = B->block == MX_BLOCK_2D;
  a.M = M;
  a.N = N;
  a.K = A->K;
  a.codes = out->codes;
  a.scales = out->scales;
  a.ld_codes = out->ld_codes;
  a.ld_scales = out->ld_scales;
  a.scale_mode = scale_mode;
  a.a_elem = A->elem;
  a.b_elem = B->elem;
  if (!mx::gemm_quantize_supported(a))
    return fail(MX_ERR_UNSUPPORTED,
                "mx_gemm_quantize: needs M, N >= 256, operand scale rows 16-byte aligned with strides %% 16 == 0, "
                "operands under 2 GiB, out code rows 4-byte aligned");
  return hip_status(mx::launch_gemm_quantize(a, static_cast<hipStream_t>(stream)), "mx_gemm_quantize");
}

mx_status mx_grouped_gemm_quantize(const mx_tensor* A, const int32_t* d_group_offsets, int32_t E,
                                   const mx_tensor* B, int64_t expert_stride_codes, int64_t expert_stride_scales,
                                   int32_t scale_mode, mx_tensor* out, void* stream) {
  g_err[0] = '\0';
  mx_status st = check_tensor(A, "mx_grouped_gemm_quantize: A");
  if (st != MX_OK) return st;
  st = check_tensor(B, "mx_grouped_gemm_quantize: B");
  if (st != MX_OK) return st;
  st = check_tensor(out, "mx_grouped_gemm_quantize: out");
  if (st != MX_OK) return st;
  if (A->block != MX_BLOCK_1D) return fail(MX_ERR_UNSUPPORTED, "mx_grouped_gemm_quantize: A must use 1-D blocks");
  if (A->K != B->K)
    return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm_quantize: A.K=%lld != B.K=%lld", (long long)A->K,
                (long long)B->K);
  if (E < 1) return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm_quantize: E=%d < 1", E);
  if (!d_group_offsets) return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm_quantize: null group offsets");
  if (scale_mode < MX_SCALE_FLOOR || scale_mode > MX_SCALE_PRESCALE_3_4)
    return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm_quantize: unknown scale mode %d", scale_mode);
  if (expert_stride_codes < 0 || expert_stride_scales < 0 || expert_stride_codes % 16)
    return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm_quantize: expert strides must be >= 0 (codes stride %% 16 == 0)");
  const int64_t M = A->rows, N = B->rows;
  if (out->rows != M || out->K != N)
    return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm_quantize: out is [%lld, %lld], the product is [%lld, %lld]",
                (long long)out->rows, (long long)out->K, (long long)M, (long long)N);
  if (out->elem != MX_ELEM_E2M1) return fail(MX_ERR_UNSUPPORTED, "mx_grouped_gemm_quantize: the output is MXFP4");
  if ((A->elem == MX_ELEM_E2M1) != (B->elem == MX_ELEM_E2M1))
    return fail(MX_ERR_UNSUPPORTED, "mx_grouped_gemm_quantize: both operands MXFP4, or both MXFP8 / MXFP6");
  if (out->block != MX_BLOCK_1D)
    return fail(MX_ERR_UNSUPPORTED, "mx_grouped_gemm_quantize: the output uses 1-D blocks");
  if (M == 0 || N == 0) return MX_OK;
  mx::GroupedQuantArgs q{};
  q.g.A = operand(A);
  q.g.B = operand(B);
  q.g.a_2d = false;
  q.g.b_2d = B->block == MX_BLOCK_2D;
  q.g.M_cap = M;
  q.g.N = N;
  q.g.K = A->K;
  q.g.offsets = d_group_offsets;
  q.g.E = E;
  q.g.stride_codes = expert_stride_codes;
  q.g.stride_scales = expert_stride_scales;
  q.codes = out->codes;
  q.scales = out->scales;
  q.ld_codes = out->ld_codes;
  q.ld_scales = out->ld_scales;
  q.scale_mode = scale_mode;
  q.g.a_elem = A->elem;
  q.g.b_elem = B->elem;
  if (!mx::grouped_quantize_supported(q))
    return fail(MX_ERR_UNSUPPORTED,
                "mx_grouped_gemm_quantize: needs N >= 256, 16-byte aligned scale rows with strides %% 16 == 0 (and "
                "expert scale stride), E <= 960, operands under 2 GiB");
  return hip_status(mx::launch_grouped_gemm_quantize(q, static_cast<hipStream_t>(stream)),
                    "mx_grouped_gemm_quantize");
}

mx_status mx_grouped_gemm(const mx_tensor* A, const int32_t* d_group_offsets, int32_t E,
                          const mx_tensor* B, int64_t expert_stride_codes,
                          int64_t expert_stride_scales, void* C, int32_t c_dtype, int64_t ldc,
                          void* stream) {
  g_err[0] = '\0';
  mx_status st = check_tensor(A, "mx_grouped_gemm: A");
  if (st != MX_OK) return st;
  st = check_tensor(B, "mx_grouped_gemm: B");
  if (st != MX_OK) return st;
  if (A->block != MX_BLOCK_1D)
    return fail(MX_ERR_UNSUPPORTED, "mx_grouped_gemm: A must use 1-D blocks (expert boundaries are arbitrary rows)");
  if (A->K != B->K)
    return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm: A.K=%lld != B.K=%lld", (long long)A->K, (long long)B->K);
  if (E < 1) return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm: E=%d < 1", E);
  if (!d_group_offsets) return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm: null group offsets");
  if (c_dtype != MX_DT_F32 && c_dtype != MX_DT_BF16)
    return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm: unknown output dtype %d", c_dtype);
  if (expert_stride_codes < 0 || expert_stride_scales < 0 || expert_stride_codes % 16)
    return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm: expert strides must be >= 0 (codes stride %% 16 == 0)");
  const int64_t M = A->rows, N = B->rows;
  if (M == 0 || N == 0) return MX_OK;
  if (!C) return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm: null C");
  if (ldc < N) return fail(MX_ERR_INVALID_ARG, "mx_grouped_gemm: ldc=%lld < N=%lld", (long long)ldc, (long long)N);
  if ((M + 127) / 128 + E > 65535) return fail(MX_ERR_UNSUPPORTED, "mx_grouped_gemm: too many row tiles");
  if (((M + 255) / 256 + E) * ((N + 255) / 256) > 0x7FFFFFFF)
    return fail(MX_ERR_UNSUPPORTED, "mx_grouped_gemm: too many tiles");
  mx::GroupedGemmArgs a{};
  a.A = operand(A);
  a.B = operand(B);
  a.a_2d = false;
  a.b_2d = B->block == MX_BLOCK_2D;
  a.M_cap = M;
  a.N = N;
  a.K = A->K;
  a.offsets = d_group_offsets;
  a.E = E;
  a.stride_codes = expert_stride_codes;
  a.stride_scales = expert_stride_scales;
  a.C = C;
  a.ldc = ldc;
  a.out_bf16 = c_dtype == MX_DT_BF16;
  a.a_elem = A->elem;
  a.b_elem = B->elem;
  if ((a.a_elem != 0 || a.b_elem != 0) &&
      !(tile_offsets_fit(A, ldc * (a.out_bf16 ? 2 : 4)) && tile_offsets_fit(B, 0)))
    return fail(MX_ERR_UNSUPPORTED, "mx_grouped_gemm: row strides too large for the MXFP8/MXFP6 kernels");
  return hip_status(mx::launch_grouped_gemm(a, static_cast<hipStream_t>(stream)), "mx_grouped_gemm");
}


// ---------------------------------------------------------------- feed-forward block
namespace {

bool known_dtype(int32_t d) { return d == MX_DT_F32 || d == MX_DT_BF16; }
uintptr_t dtype_size(int32_t d) { return d == MX_DT_BF16 ? 2 : 4; }

// A row-major [R, C] buffer of `dtype` elements, element-aligned.
mx_status check_rows(const void* p, int32_t dtype, int64_t C, int64_t ld, const char* what, const char* name) {
  if (!p) return fail(MX_ERR_INVALID_ARG, "%s: null %s", what, name);
  if (ld < C)
    return fail(MX_ERR_INVALID_ARG, "%s: row stride of %s %lld < %lld", what, name, (long long)ld, (long long)C);
  if (!aligned(p, dtype_size(dtype)))
    return fail(MX_ERR_INVALID_ARG, "%s: %s must be aligned to its element size", what, name);
  return MX_OK;
}

// Validate a gated block's operands and configuration and describe them; the
// buffers follow.  M = 0 or N = 0 leaves a.M or a.N 0.
mx_status gated_args(const mx_tensor* A, const mx_tensor* B, const mx_gate_cfg* cfg, const char* what,
                     mx::GatedArgs& a) {
  char name[64];
  std::snprintf(name, sizeof(name), "%s: A", what);
  mx_status st = check_tensor(A, name);
  if (st != MX_OK) return st;
  std::snprintf(name, sizeof(name), "%s: B", what);
  st = check_tensor(B, name);
  if (st != MX_OK) return st;
  if (A->K != B->K)
    return fail(MX_ERR_INVALID_ARG, "%s: A.K=%lld != B.K=%lld", what, (long long)A->K, (long long)B->K);
  if (B->rows % 2)
    return fail(MX_ERR_INVALID_ARG, "%s: B holds gate and up rows, an even number (got %lld)", what,
                (long long)B->rows);
  if (!cfg) return fail(MX_ERR_INVALID_ARG, "%s: null gate configuration", what);
  if (cfg->act < MX_ACT_SILU || cfg->act > MX_ACT_GELU_TANH)
    return fail(MX_ERR_INVALID_ARG, "%s: unknown activation %d", what, cfg->act);
  if (cfg->layout != MX_GATE_INTERLEAVED && cfg->layout != MX_GATE_HALVES)
    return fail(MX_ERR_INVALID_ARG, "%s: unknown gate layout %d", what, cfg->layout);
  if (!(cfg->alpha > 0.0f) || !std::isfinite(cfg->alpha))
    return fail(MX_ERR_INVALID_ARG, "%s: alpha must be finite and > 0", what);
  if (!(cfg->limit >= 0.0f)) return fail(MX_ERR_INVALID_ARG, "%s: limit must be >= 0 (0: none)", what);
  if (!std::isfinite(cfg->up_shift)) return fail(MX_ERR_INVALID_ARG, "%s: up_shift must be finite", what);
  if (A->rows > 0x7FFFFFFF || B->rows > 0x7FFFFFFF || A->K > 0x7FFFFFFF)
    return fail(MX_ERR_UNSUPPORTED, "%s: at most 2^31 - 1 rows and K elements", what);
  a = mx::GatedArgs{};
  a.A = operand(A);
  a.B = operand(B);
  a.a_2d = A->block == MX_BLOCK_2D;
  a.b_2d = B->block == MX_BLOCK_2D;
  a.a_elem = A->elem;
  a.b_elem = B->elem;
  a.M = A->rows;
  a.N = B->rows / 2;
  a.K = A->K;
  a.act = cfg->act;
  a.halves = cfg->layout == MX_GATE_HALVES;
  a.alpha = cfg->alpha;
  a.limit = cfg->limit == 0.0f ? INFINITY : cfg->limit;
  a.up_shift = cfg->up_shift;
  return MX_OK;
}

// The output of the forward pass (dH null) or the backward pass's two buffers.
mx_status gated_buffers(mx::GatedArgs& a, bool backward, const void* dH, int32_t dh_dtype, int64_t lddh, void* out,
                        int32_t out_dtype, int64_t ldo, const char* what) {
  if (!known_dtype(out_dtype)) return fail(MX_ERR_INVALID_ARG, "%s: unknown output dtype %d", what, out_dtype);
  if (backward && !known_dtype(dh_dtype)) return fail(MX_ERR_INVALID_ARG, "%s: unknown dH dtype %d", what, dh_dtype);
  if (a.M == 0 || a.N == 0) return MX_OK;
  mx_status st = check_rows(out, out_dtype, backward ? 2 * a.N : a.N, ldo, what, backward ? "dP" : "H");
  if (st != MX_OK) return st;
  a.out = out;
  a.ldo = ldo;
  a.out_bf16 = out_dtype == MX_DT_BF16;
  if (backward) {
    st = check_rows(dH, dh_dtype, a.N, lddh, what, "dH");
    if (st != MX_OK) return st;
    a.dH = dH;
    a.lddh = lddh;
    a.dh_bf16 = dh_dtype == MX_DT_BF16;
  }
  return MX_OK;
}

mx_status gated_groups(mx::GatedArgs& a, const mx_tensor* A, const int32_t* offsets, int32_t E, int64_t stride_codes,
                       int64_t stride_scales, const char* what) {
  if (A->block != MX_BLOCK_1D)
    return fail(MX_ERR_UNSUPPORTED, "%s: A must use 1-D blocks (expert boundaries are arbitrary rows)", what);
  if (E < 1) return fail(MX_ERR_INVALID_ARG, "%s: E=%d < 1", what, E);
  if (!offsets || !aligned(offsets, 4)) return fail(MX_ERR_INVALID_ARG, "%s: null or unaligned group offsets", what);
  if (stride_codes < 0 || stride_scales < 0 || stride_codes % 16)
    return fail(MX_ERR_INVALID_ARG, "%s: expert strides must be >= 0 (codes stride %% 16 == 0)", what);
  a.offsets = offsets;
  a.E = E;
  a.stride_codes = stride_codes;
  a.stride_scales = stride_scales;
  return MX_OK;
}

}  // namespace

mx_status mx_gemm_gated(const mx_tensor* A, const mx_tensor* B, const mx_gate_cfg* cfg, void* H, int32_t h_dtype,
                        int64_t ldh, void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_gemm_gated";
  mx::GatedArgs a;
  mx_status st = gated_args(A, B, cfg, what, a);
  if (st == MX_OK) st = gated_buffers(a, false, nullptr, 0, 0, H, h_dtype, ldh, what);
  if (st != MX_OK) return st;
  return hip_status(mx::launch_gated(a, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_gemm_gated_backward(const mx_tensor* A, const mx_tensor* B, const mx_gate_cfg* cfg, const void* dH,
                                 int32_t dh_dtype, int64_t lddh, void* dP, int32_t dp_dtype, int64_t lddp,
                                 void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_gemm_gated_backward";
  mx::GatedArgs a;
  mx_status st = gated_args(A, B, cfg, what, a);
  if (st == MX_OK) st = gated_buffers(a, true, dH, dh_dtype, lddh, dP, dp_dtype, lddp, what);
  if (st != MX_OK) return st;
  return hip_status(mx::launch_gated(a, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_grouped_gemm_gated(const mx_tensor* A, const int32_t* d_group_offsets, int32_t E, const mx_tensor* B,
                                int64_t expert_stride_codes, int64_t expert_stride_scales, const mx_gate_cfg* cfg,
                                void* H, int32_t h_dtype, int64_t ldh, void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_grouped_gemm_gated";
  mx::GatedArgs a;
  mx_status st = gated_args(A, B, cfg, what, a);
  if (st == MX_OK) st = gated_groups(a, A, d_group_offsets, E, expert_stride_codes, expert_stride_scales, what);
  if (st == MX_OK) st = gated_buffers(a, false, nullptr, 0, 0, H, h_dtype, ldh, what);
  if (st != MX_OK) return st;
  return hip_status(mx::launch_gated(a, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_grouped_gemm_gated_backward(const mx_tensor* A, const int32_t* d_group_offsets, int32_t E,
                                         const mx_tensor* B, int64_t expert_stride_codes,
                                         int64_t expert_stride_scales, const mx_gate_cfg* cfg, const void* dH,
                                         int32_t dh_dtype, int64_t lddh, void* dP, int32_t dp_dtype, int64_t lddp,
                                         void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_grouped_gemm_gated_backward";
  mx::GatedArgs a;
  mx_status st = gated_args(A, B, cfg, what, a);
  if (st == MX_OK) st = gated_groups(a, A, d_group_offsets, E, expert_stride_codes, expert_stride_scales, what);
  if (st == MX_OK) st = gated_buffers(a, true, dH, dh_dtype, lddh, dP, dp_dtype, lddp, what);
  if (st != MX_OK) return st;
  return hip_status(mx::launch_gated(a, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_layer_norm(const void* x, int32_t dtype, int64_t R, int64_t C, int64_t ldx, const void* weight,
                        const void* bias, int32_t w_dtype, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                        void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_layer_norm";
  if (!known_dtype(dtype)) return fail(MX_ERR_INVALID_ARG, "%s: unknown dtype %d", what, dtype);
  if (!known_dtype(w_dtype)) return fail(MX_ERR_INVALID_ARG, "%s: unknown weight dtype %d", what, w_dtype);
  if (R < 0 || C < 0) return fail(MX_ERR_INVALID_ARG, "%s: negative shape", what);
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(MX_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", what);
  if (R == 0 || C == 0) return MX_OK;
  mx_status st = check_rows(x, dtype, C, ldx, what, "x");
  if (st == MX_OK) st = check_rows(y, dtype, C, ldy, what, "y");
  if (st != MX_OK) return st;
  if (!aligned(weight, dtype_size(w_dtype)) || !aligned(bias, dtype_size(w_dtype)))
    return fail(MX_ERR_INVALID_ARG, "%s: weight and bias must be aligned to their element size", what);
  if (!aligned(mean, 4) || !aligned(rstd, 4))
    return fail(MX_ERR_INVALID_ARG, "%s: mean and rstd must be 4-byte aligned", what);
  mx::NormArgs a{};
  a.x = x;
  a.R = R;
  a.C = C;
  a.ldx = ldx;
  a.bf16 = dtype == MX_DT_BF16;
  a.weight = weight;
  a.bias = bias;
  a.w_bf16 = w_dtype == MX_DT_BF16;
  a.eps = eps;
  a.y = y;
  a.ldy = ldy;
  a.mean = mean;
  a.rstd = rstd;
  return hip_status(mx::launch_layer_norm(a, static_cast<hipStream_t>(stream)), what);
}

size_t mx_layer_norm_backward_workspace_size(int64_t R, int64_t C) {
  if (R <= 0 || C <= 0) return 0;
  return mx::norm_backward_workspace(R, C);
}

mx_status mx_layer_norm_backward(const void* dy, const void* x, int32_t dtype, int64_t R, int64_t C, int64_t lddy,
                                 int64_t ldx, const float* mean, const float* rstd, const void* weight,
                                 int32_t w_dtype, void* dx, int64_t lddx, void* dweight, void* dbias, void* workspace,
                                 size_t ws_bytes, void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_layer_norm_backward";
  if (!known_dtype(dtype)) return fail(MX_ERR_INVALID_ARG, "%s: unknown dtype %d", what, dtype);
  if (!known_dtype(w_dtype)) return fail(MX_ERR_INVALID_ARG, "%s: unknown weight dtype %d", what, w_dtype);
  if (R < 0 || C < 0) return fail(MX_ERR_INVALID_ARG, "%s: negative shape", what);
  if (C == 0) return MX_OK;
  const uintptr_t ws = dtype_size(w_dtype);
  if (!aligned(weight, ws) || !aligned(dweight, ws) || !aligned(dbias, ws))
    return fail(MX_ERR_INVALID_ARG, "%s: weight, dweight and dbias must be aligned to their element size", what);
  if (R > 0) {
    mx_status st = check_rows(dy, dtype, C, lddy, what, "dy");
    if (st == MX_OK) st = check_rows(x, dtype, C, ldx, what, "x");
    if (st == MX_OK && dx) st = check_rows(dx, dtype, C, lddx, what, "dx");
    if (st != MX_OK) return st;
    if (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4))
      return fail(MX_ERR_INVALID_ARG, "%s: null or unaligned mean or rstd", what);
    if (dweight || dbias) {
      const size_t need = mx::norm_backward_workspace(R, C);
      if (!workspace || ws_bytes < need || !aligned(workspace, 16))
        return fail(MX_ERR_INVALID_ARG,
                    "%s: dweight and dbias need a 16-byte aligned workspace of %zu bytes (got %zu bytes at %p)", what,
                    need, ws_bytes, workspace);
    }
  }
  mx::NormBwdArgs a{};
  a.dy = dy;
  a.x = x;
  a.R = R;
  a.C = C;
  a.lddy = lddy;
  a.ldx = ldx;
  a.bf16 = dtype == MX_DT_BF16;
  a.mean = mean;
  a.rstd = rstd;
  a.weight = weight;
  a.w_bf16 = w_dtype == MX_DT_BF16;
  a.dx = dx;
  a.lddx = lddx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.workspace = static_cast<float*>(workspace);
  return hip_status(mx::launch_layer_norm_backward(a, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_dropout(const void* x, int32_t dtype, int64_t R, int64_t C, int64_t ldx, float p, uint64_t seed,
                     uint64_t offset, const void* residual, int64_t ldr, void* y, int64_t ldy, void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_dropout";
  if (!known_dtype(dtype)) return fail(MX_ERR_INVALID_ARG, "%s: unknown dtype %d", what, dtype);
  if (R < 0 || C < 0) return fail(MX_ERR_INVALID_ARG, "%s: negative shape", what);
  if (!(p >= 0.0f && p <= 1.0f)) return fail(MX_ERR_INVALID_ARG, "%s: p must be in [0, 1]", what);
  if (R == 0 || C == 0) return MX_OK;
  mx_status st = check_rows(x, dtype, C, ldx, what, "x");
  if (st == MX_OK) st = check_rows(y, dtype, C, ldy, what, "y");
  if (st == MX_OK && residual) st = check_rows(residual, dtype, C, ldr, what, "residual");
  if (st != MX_OK) return st;
  mx::DropoutArgs a{};
  a.x = x;
  a.residual = residual;
  a.y = y;
  a.R = R;
  a.C = C;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldy;
  a.bf16 = dtype == MX_DT_BF16;
  a.threshold = (uint32_t)std::nearbyint((double)p * 65536.0);
  a.seed = seed;
  a.offset = offset;
  return hip_status(mx::launch_dropout(a, static_cast<hipStream_t>(stream)), what);
}

// ---------------------------------------------------------------- expert layer
namespace {

constexpr int32_t EXPERTS_MAX = 1024, CHOICES_MAX = 64;
constexpr int64_t WAVES_MAX = (1 << 26) - 4;   // a launch has fewer than 2^32 threads, 256 per workgroup

mx_status router_args(const void* logits, int32_t dtype, int64_t T, int32_t E, int64_t ld, int32_t top,
                      const mx_router_cfg* cfg, const char* what, mx::RouteArgs& a) {
  if (!known_dtype(dtype)) return fail(MX_ERR_INVALID_ARG, "%s: unknown dtype %d", what, dtype);
  if (!cfg) return fail(MX_ERR_INVALID_ARG, "%s: null router configuration", what);
  if (cfg->score != MX_SCORE_SOFTMAX && cfg->score != MX_SCORE_SIGMOID)
    return fail(MX_ERR_INVALID_ARG, "%s: unknown score %d", what, cfg->score);
  if (cfg->renormalize != 0 && cfg->renormalize != 1)
    return fail(MX_ERR_INVALID_ARG, "%s: renormalize must be 0 or 1", what);
  if (!std::isfinite(cfg->scale)) return fail(MX_ERR_INVALID_ARG, "%s: scale must be finite", what);
  if (T < 0) return fail(MX_ERR_INVALID_ARG, "%s: negative shape", what);
  if (E < 1) return fail(MX_ERR_INVALID_ARG, "%s: E=%d < 1", what, E);
  if (top < 1 || top > E) return fail(MX_ERR_INVALID_ARG, "%s: top=%d is not in 1 .. E=%d", what, top, E);
  if (E > EXPERTS_MAX || top > CHOICES_MAX || T > WAVES_MAX)
    return fail(MX_ERR_UNSUPPORTED, "%s: at most %d experts, %d choices and 2^26 - 4 tokens", what, EXPERTS_MAX,
                CHOICES_MAX);
  if (T == 0) return MX_OK;
  mx_status st = check_rows(logits, dtype, E, ld, what, "logits");
  if (st != MX_OK) return st;
  a = mx::RouteArgs{};
  a.logits = logits;
  a.T = T;
  a.ld = ld;
  a.E = E;
  a.top = top;
  a.bf16 = dtype == MX_DT_BF16;
  a.sigmoid = cfg->score == MX_SCORE_SIGMOID;
  a.renorm = cfg->renormalize == 1;
  a.scale = cfg->scale;
  return MX_OK;
}

mx_status check_words(const void* p, const char* what, const char* name) {
  if (!p || !aligned(p, 4)) return fail(MX_ERR_INVALID_ARG, "%s: null or unaligned %s", what, name);
  return MX_OK;
}

// The shape of a dispatch or combine: T tokens of `top` choices, `rows` sorted
// rows, C columns.
mx_status combine_args(int32_t dtype, int64_t T, int64_t C, int64_t rows, int32_t top, const int32_t* dest,
                       const char* what, mx::CombineArgs& a) {
  if (!known_dtype(dtype)) return fail(MX_ERR_INVALID_ARG, "%s: unknown dtype %d", what, dtype);
  if (T < 0 || C < 0 || rows < 0) return fail(MX_ERR_INVALID_ARG, "%s: negative shape", what);
  if (top < 1) return fail(MX_ERR_INVALID_ARG, "%s: top=%d < 1", what, top);
  // (at most a wave per 64 pieces of 16 bytes of a row, and for a row)
  const int64_t piece = 64 * 16 / (int64_t)dtype_size(dtype);
  if (T > WAVES_MAX || C > 0x7FFFFFFF || T * ((C + piece - 1) / piece) > WAVES_MAX)
    return fail(MX_ERR_UNSUPPORTED, "%s: too many rows or columns", what);
  if (T && C) {
    mx_status st = check_words(dest, what, "dest");
    if (st != MX_OK) return st;
  }
  a = mx::CombineArgs{};
  a.T = T;
  a.C = C;
  a.rows = rows;
  a.top = top;
  a.bf16 = dtype == MX_DT_BF16;
  a.dest = dest;
  return MX_OK;
}

}  // namespace

mx_status mx_route(const void* logits, int32_t dtype, int64_t T, int32_t E, int64_t ld, int32_t top,
                   const mx_router_cfg* cfg, int32_t* ids, float* weights, void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_route";
  mx::RouteArgs a;
  mx_status st = router_args(logits, dtype, T, E, ld, top, cfg, what, a);
  if (st != MX_OK || T == 0) return st;
  st = check_words(ids, what, "ids");
  if (st == MX_OK) st = check_words(weights, what, "weights");
  if (st != MX_OK) return st;
  a.ids = ids;
  a.weights = weights;
  return hip_status(mx::launch_route(a, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_route_backward(const float* dweights, const void* logits, int32_t dtype, int64_t T, int32_t E, int64_t ld,
                            const int32_t* ids, int32_t top, const mx_router_cfg* cfg, void* dlogits, int64_t ldd,
                            void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_route_backward";
  mx::RouteArgs a;
  mx_status st = router_args(logits, dtype, T, E, ld, top, cfg, what, a);
  if (st != MX_OK || T == 0) return st;
  st = check_words(ids, what, "ids");
  if (st == MX_OK) st = check_words(dweights, what, "dweights");
  if (st == MX_OK) st = check_rows(dlogits, dtype, E, ldd, what, "dlogits");
  if (st != MX_OK) return st;
  a.ids = const_cast<int32_t*>(ids);
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.ldd = ldd;
  return hip_status(mx::launch_route(a, static_cast<hipStream_t>(stream)), what);
}

size_t mx_expert_sort_workspace_size(int64_t T, int32_t top, int32_t E) {
  if (T <= 0 || top < 1 || E < 1 || E > EXPERTS_MAX || T > 0x7FFFFFFF / top) return 0;
  return mx::sort_workspace(T * top, E);
}

mx_status mx_expert_sort(const int32_t* ids, int64_t T, int32_t top, int32_t E, int32_t* offsets, int32_t* rows,
                         int32_t* dest, void* workspace, size_t ws_bytes, void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_expert_sort";
  if (T < 0) return fail(MX_ERR_INVALID_ARG, "%s: negative shape", what);
  if (top < 1) return fail(MX_ERR_INVALID_ARG, "%s: top=%d < 1", what, top);
  if (E < 1) return fail(MX_ERR_INVALID_ARG, "%s: E=%d < 1", what, E);
  if (E > EXPERTS_MAX || T > 0x7FFFFFFF / top)
    return fail(MX_ERR_UNSUPPORTED, "%s: at most %d experts and 2^31 - 1 slots", what, EXPERTS_MAX);
  mx_status st = check_words(offsets, what, "offsets");
  if (st == MX_OK && T) st = check_words(ids, what, "ids");
  if (st == MX_OK && T) st = check_words(rows, what, "rows");
  if (st == MX_OK && T) st = check_words(dest, what, "dest");
  if (st != MX_OK) return st;
  const size_t need = mx::sort_workspace(T * top, E);
  if (need && (!workspace || ws_bytes < need || !aligned(workspace, 4)))
    return fail(MX_ERR_INVALID_ARG, "%s: needs a 4-byte aligned workspace of %zu bytes (got %zu bytes at %p)", what,
                need, ws_bytes, workspace);
  mx::SortArgs a{};
  a.ids = ids;
  a.n = T * top;
  a.top = top;
  a.E = E;
  a.offsets = offsets;
  a.rows = rows;
  a.dest = dest;
  a.ws = static_cast<int*>(workspace);
  return hip_status(mx::launch_expert_sort(a, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_expert_dispatch(const void* x, int32_t dtype, int64_t T, int64_t C, int64_t ldx, const int32_t* dest,
                             int32_t top, void* xs, int64_t rows, int64_t ldxs, void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_expert_dispatch";
  mx::CombineArgs a;
  mx_status st = combine_args(dtype, T, C, rows, top, dest, what, a);
  if (st != MX_OK || T == 0 || C == 0 || rows == 0) return st;
  st = check_rows(x, dtype, C, ldx, what, "x");
  if (st == MX_OK) st = check_rows(xs, dtype, C, ldxs, what, "xs");
  if (st != MX_OK) return st;
  a.dout = x;
  a.lddo = ldx;
  a.dy = xs;
  a.lddy = ldxs;
  return hip_status(mx::launch_dispatch(a, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_expert_combine(const void* y, int32_t dtype, int64_t rows, int64_t C, int64_t ldy, const int32_t* dest,
                            const float* weights, int64_t T, int32_t top, const void* residual, int64_t ldr, void* out,
                            int64_t ldo, void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_expert_combine";
  mx::CombineArgs a;
  mx_status st = combine_args(dtype, T, C, rows, top, dest, what, a);
  if (st != MX_OK || T == 0 || C == 0) return st;
  if (!aligned(weights, 4)) return fail(MX_ERR_INVALID_ARG, "%s: unaligned weights", what);
  if (rows) st = check_rows(y, dtype, C, ldy, what, "y");
  if (st == MX_OK && residual) st = check_rows(residual, dtype, C, ldr, what, "residual");
  if (st == MX_OK) st = check_rows(out, dtype, C, ldo, what, "out");
  if (st != MX_OK) return st;
  a.weights = weights;
  a.y = y;
  a.ldy = ldy;
  a.residual = residual;
  a.ldr = ldr;
  a.out = out;
  a.ldo = ldo;
  if (rows == 0) a.top = 0;                  // no row to take: zeros, or the residual
  return hip_status(mx::launch_combine(a, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_expert_combine_backward(const void* dout, int32_t dtype, int64_t T, int64_t C, int64_t lddo,
                                     const void* y, int64_t rows, int64_t ldy, const int32_t* dest,
                                     const float* weights, int32_t top, void* dy, int64_t lddy, float* dweights,
                                     void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_expert_combine_backward";
  mx::CombineArgs a;
  mx_status st = combine_args(dtype, T, C, rows, top, dest, what, a);
  if (st != MX_OK || T == 0) return st;
  // (without rows or columns every dweight is still a sum, of nothing)
  st = check_words(dest, what, "dest");
  if (st == MX_OK) st = check_words(weights, what, "weights");
  if (st == MX_OK) st = check_words(dweights, what, "dweights");
  if (st == MX_OK && C && rows) st = check_rows(dout, dtype, C, lddo, what, "dout");
  if (st == MX_OK && C && rows) st = check_rows(y, dtype, C, ldy, what, "y");
  if (st == MX_OK && C && rows) st = check_rows(dy, dtype, C, lddy, what, "dy");
  if (st != MX_OK) return st;
  if (rows == 0) a.C = 0;                    // nothing may be read
  a.dout = dout;
  a.lddo = lddo;
  a.y = y;
  a.ldy = ldy;
  a.weights = weights;
  a.dy = dy;
  a.lddy = lddy;
  a.dweights = dweights;
  return hip_status(mx::launch_combine_backward(a, static_cast<hipStream_t>(stream)), what);
}

namespace {

mx_status bias_grad(const void* dp, int32_t dtype, int64_t M, int64_t N, int64_t ld, bool grouped,
                    const int32_t* offsets, int32_t E, void* out, int32_t out_dtype, void* workspace, size_t ws_bytes,
                    void* stream, const char* what) {
  if (!known_dtype(dtype)) return fail(MX_ERR_INVALID_ARG, "%s: unknown dtype %d", what, dtype);
  if (!known_dtype(out_dtype)) return fail(MX_ERR_INVALID_ARG, "%s: unknown output dtype %d", what, out_dtype);
  if (M < 0 || N < 0) return fail(MX_ERR_INVALID_ARG, "%s: negative shape", what);
  if (E < 1) return fail(MX_ERR_INVALID_ARG, "%s: E=%d < 1", what, E);
  if (grouped) {
    mx_status st = check_words(offsets, what, "group offsets");
    if (st != MX_OK) return st;
  }
  if (N == 0) return MX_OK;
  if (M > 0x7FFFFFFF || N > 0x7FFFFFFF || !mx::bias_grad_fits(M, N, E, grouped))
    return fail(MX_ERR_UNSUPPORTED, "%s: too many rows or columns", what);
  if (!out || !aligned(out, dtype_size(out_dtype)))
    return fail(MX_ERR_INVALID_ARG, "%s: null out, or not aligned to its element size", what);
  if (M) {
    mx_status st = check_rows(dp, dtype, N, ld, what, "dp");
    if (st != MX_OK) return st;
  }
  const size_t need = mx::bias_grad_workspace(M, N, E, grouped);
  if (need && (!workspace || ws_bytes < need || !aligned(workspace, 4)))
    return fail(MX_ERR_INVALID_ARG, "%s: needs a 4-byte aligned workspace of %zu bytes (got %zu bytes at %p)", what,
                need, ws_bytes, workspace);
  mx::BiasGradArgs a{};
  a.dp = dp;
  a.M = M;
  a.N = N;
  a.ld = ld;
  a.bf16 = dtype == MX_DT_BF16;
  a.offsets = offsets;
  a.E = E;
  a.out = out;
  a.out_bf16 = out_dtype == MX_DT_BF16;
  a.ws = static_cast<float*>(workspace);
  return hip_status(mx::launch_bias_grad(a, static_cast<hipStream_t>(stream)), what);
}

}  // namespace

size_t mx_bias_grad_workspace_size(int64_t M, int64_t N, int32_t E) {
  if (M <= 0 || N <= 0 || E < 1 || M > 0x7FFFFFFF || N > 0x7FFFFFFF) return 0;
  return mx::bias_grad_workspace(M, N, E, true);     // (a grouped call's, no less than a dense one's)
}

mx_status mx_bias_grad(const void* dp, int32_t dtype, int64_t M, int64_t N, int64_t ld, void* out, int32_t out_dtype,
                       void* workspace, size_t ws_bytes, void* stream) {
  g_err[0] = '\0';
  return bias_grad(dp, dtype, M, N, ld, false, nullptr, 1, out, out_dtype, workspace, ws_bytes, stream, "mx_bias_grad");
}

mx_status mx_grouped_bias_grad(const void* dp, int32_t dtype, int64_t M, int64_t N, int64_t ld,
                               const int32_t* d_group_offsets, int32_t E, void* out, int32_t out_dtype, void* workspace,
                               size_t ws_bytes, void* stream) {
  g_err[0] = '\0';
  return bias_grad(dp, dtype, M, N, ld, true, d_group_offsets, E, out, out_dtype, workspace, ws_bytes, stream,
                   "mx_grouped_bias_grad");
}

// ---------------------------------------------------------------- linear layer
namespace {

struct Buffer {
  const void* p;
  int32_t dtype;
  int64_t ld;
};

// Validate a linear layer's operands, epilogue and buffers and describe them: r is the
// residual (p null: none) or, backward, dY.
mx_status linear_args(const mx_tensor* A, const mx_tensor* B, const mx_epilogue_cfg* cfg, const void* bias,
                      int32_t bias_dtype, int64_t bias_stride, bool backward, const Buffer& r, const Buffer& out,
                      const char* what, mx::LinearArgs& a) {
  char name[64];
  std::snprintf(name, sizeof(name), "%s: A", what);
  mx_status st = check_tensor(A, name);
  if (st != MX_OK) return st;
  std::snprintf(name, sizeof(name), "%s: B", what);
  st = check_tensor(B, name);
  if (st != MX_OK) return st;
  if (A->K != B->K)
    return fail(MX_ERR_INVALID_ARG, "%s: A.K=%lld != B.K=%lld", what, (long long)A->K, (long long)B->K);
  const int32_t act = cfg ? cfg->act : (int32_t)MX_ACT_NONE;
  if (act < MX_ACT_SILU || act > MX_ACT_NONE) return fail(MX_ERR_INVALID_ARG, "%s: unknown activation %d", what, act);
  if (act == MX_ACT_SILU && (!(cfg->alpha > 0.0f) || !std::isfinite(cfg->alpha)))   // (the others ignore it)
    return fail(MX_ERR_INVALID_ARG, "%s: alpha must be finite and > 0", what);
  if (backward && act == MX_ACT_NONE)
    return fail(MX_ERR_INVALID_ARG, "%s: without an activation the gradient is dY itself", what);
  if (!known_dtype(out.dtype)) return fail(MX_ERR_INVALID_ARG, "%s: unknown output dtype %d", what, out.dtype);
  if (bias && !known_dtype(bias_dtype))
    return fail(MX_ERR_INVALID_ARG, "%s: unknown bias dtype %d", what, bias_dtype);
  if ((r.p || backward) && !known_dtype(r.dtype))
    return fail(MX_ERR_INVALID_ARG, "%s: unknown %s dtype %d", what, backward ? "dY" : "residual", r.dtype);
  if (A->rows > 0x7FFFFFFF || B->rows > 0x7FFFFFFF || A->K > 0x7FFFFFFF)
    return fail(MX_ERR_UNSUPPORTED, "%s: at most 2^31 - 1 rows and K elements", what);
  a = mx::LinearArgs{};
  a.A = operand(A);
  a.B = operand(B);
  a.a_2d = A->block == MX_BLOCK_2D;
  a.b_2d = B->block == MX_BLOCK_2D;
  a.a_elem = A->elem;
  a.b_elem = B->elem;
  a.M = A->rows;
  a.N = B->rows;
  a.K = A->K;
  a.act = act;
  a.alpha = act == MX_ACT_SILU ? cfg->alpha : 1.0f;
  a.backward = backward;
  if (a.M == 0 || a.N == 0) return MX_OK;
  st = check_rows(out.p, out.dtype, a.N, out.ld, what, backward ? "dP" : "Y");
  if (st == MX_OK && (r.p || backward)) st = check_rows(r.p, r.dtype, a.N, r.ld, what, backward ? "dY" : "residual");
  if (st != MX_OK) return st;
  if (bias && (!aligned(bias, dtype_size(bias_dtype)) || bias_stride < 0))
    return fail(MX_ERR_INVALID_ARG, "%s: bias must be aligned to its element size, its stride >= 0", what);
  a.out = const_cast<void*>(out.p);
  a.ldo = out.ld;
  a.out_bf16 = out.dtype == MX_DT_BF16;
  a.dH = r.p;
  a.lddh = r.p ? r.ld : 0;
  a.dh_bf16 = r.p && r.dtype == MX_DT_BF16;
  a.bias = bias;
  a.bias_bf16 = bias && bias_dtype == MX_DT_BF16;
  a.bias_stride = bias ? bias_stride : 0;
  return MX_OK;
}

}  // namespace

mx_status mx_linear(const mx_tensor* A, const mx_tensor* B, const mx_epilogue_cfg* cfg, const void* bias,
                    int32_t bias_dtype, const void* residual, int32_t r_dtype, int64_t ldr, void* Y, int32_t y_dtype,
                    int64_t ldy, void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_linear";
  mx::LinearArgs a;
  mx_status st = linear_args(A, B, cfg, bias, bias_dtype, 0, false, {residual, r_dtype, ldr}, {Y, y_dtype, ldy}, what, a);
  if (st != MX_OK) return st;
  return hip_status(mx::launch_linear(a, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_linear_backward(const mx_tensor* A, const mx_tensor* B, const mx_epilogue_cfg* cfg, const void* bias,
                             int32_t bias_dtype, const void* dY, int32_t dy_dtype, int64_t lddy, void* dP,
                             int32_t dp_dtype, int64_t lddp, void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_linear_backward";
  mx::LinearArgs a;
  mx_status st = linear_args(A, B, cfg, bias, bias_dtype, 0, true, {dY, dy_dtype, lddy}, {dP, dp_dtype, lddp}, what, a);
  if (st != MX_OK) return st;
  return hip_status(mx::launch_linear(a, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_grouped_linear(const mx_tensor* A, const int32_t* d_group_offsets, int32_t E, const mx_tensor* B,
                            int64_t expert_stride_codes, int64_t expert_stride_scales, const mx_epilogue_cfg* cfg,
                            const void* bias, int32_t bias_dtype, int64_t bias_stride, const void* residual,
                            int32_t r_dtype, int64_t ldr, void* Y, int32_t y_dtype, int64_t ldy, void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_grouped_linear";
  mx::LinearArgs a;
  mx_status st = linear_args(A, B, cfg, bias, bias_dtype, bias_stride, false, {residual, r_dtype, ldr},
                             {Y, y_dtype, ldy}, what, a);
  if (st == MX_OK) st = gated_groups(a, A, d_group_offsets, E, expert_stride_codes, expert_stride_scales, what);
  if (st != MX_OK) return st;
  return hip_status(mx::launch_linear(a, static_cast<hipStream_t>(stream)), what);
}

mx_status mx_grouped_linear_backward(const mx_tensor* A, const int32_t* d_group_offsets, int32_t E, const mx_tensor* B,
                                     int64_t expert_stride_codes, int64_t expert_stride_scales,
                                     const mx_epilogue_cfg* cfg, const void* bias, int32_t bias_dtype,
                                     int64_t bias_stride, const void* dY, int32_t dy_dtype, int64_t lddy, void* dP,
                                     int32_t dp_dtype, int64_t lddp, void* stream) {
  g_err[0] = '\0';
  const char* what = "mx_grouped_linear_backward";
  mx::LinearArgs a;
  mx_status st = linear_args(A, B, cfg, bias, bias_dtype, bias_stride, true, {dY, dy_dtype, lddy}, {dP, dp_dtype, lddp},
                             what, a);
  if (st == MX_OK) st = gated_groups(a, A, d_group_offsets, E, expert_stride_codes, expert_stride_scales, what);
  if (st != MX_OK) return st;
  return hip_status(mx::launch_linear(a, static_cast<hipStream_t>(stream)), what);
}

}  // extern "C"
