"""MI355X-native MXFP4 (OCP MX v1.0) quantizer and block-scaled GEMMs.

A thin ctypes binding over ``libmxfp4.so`` (declared in ``include/mx.h``).
PyTorch supplies device memory and the current HIP stream; every step of the
computation runs in the library's HIP kernels.  The binding only allocates
output tensors and marshals pointers, shapes and strides.  If the library is
missing, every call raises: there is no fallback path.

    q = quantize(x, axis="last", block="1d", rounding="rne", rht_mask=None)
    y = dequantize(q, torch.float32)
    qt = transpose(q2d)                                 # exact, 2-D blocks only
    c = gemm(qa, qb, torch.bfloat16)                    # C = A * B^T
    c = grouped_gemm(qa, offsets, qb_stacked, torch.bfloat16)

and, around the products of a feed-forward block,

    h = gemm_gated(qa, qb, Gate())                      # act(gate) * up, qb = gate and up rows
    dp = gemm_gated_backward(qa, qb, dh, Gate())        # gradient of both projections
    y, mean, rstd = layer_norm(x, weight, bias)
    dx, dw, db = layer_norm_backward(dy, x, mean, rstd, weight)
    y = dropout(x, 0.1, seed=1, residual=r)
    y = linear(qa, qb, bias, act="gelu", residual=r)    # act(A * B^T + bias) + r
    dp = linear_backward(qa, qb, dy, bias, act="gelu")
    db = bias_grad(dp)

and, around the grouped products of an expert layer,

    ids, weights = route(logits, top, Router())
    offsets, rows, dest = expert_sort(ids, E)           # for grouped_*, quantize_gather, quantize_scatter
    xs = expert_dispatch(x, dest)
    ys = grouped_linear(qxs, offsets, qw, bias, act="gelu")
    y = expert_combine(ys, dest, weights, residual=x)
    dys, dweights = expert_combine_backward(dy, ys, dest, weights)
    dlogits = route_backward(dweights, logits, ids, Router())
"""
import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmxfp4.so")

MX_OK, MX_ERR_INVALID_ARG, MX_ERR_UNSUPPORTED, MX_ERR_HIP = 0, 1, 2, 3
MX_DT_F32, MX_DT_BF16 = 0, 1
_AXIS = {"last": 0, "dim0": 1}
_BLOCK = {"1d": 0, "2d": 1}
_ROUND = {"rne": 0, "sr": 1, "sr8": 2}
_SCALE = {"floor": 0, "round_up": 1, "prescale_3_4": 2}
# MX element types: name -> (mx_elem, bits per element)
_ELEM = {"e2m1": (0, 4), "e4m3": (1, 8), "e5m2": (2, 8), "e2m3": (3, 6), "e3m2": (4, 6)}
_ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
_EPILOGUE_ACT = {**_ACT, None: 3}
_SCORE = {"softmax": 0, "sigmoid": 1}
_EXPERTS_MAX, _CHOICES_MAX = 1024, 64           # of a router (mx_route in include/mx.h)
_GATE_LAYOUT = {"interleaved": 0, "halves": 1}
_DTYPE = {torch.float32: MX_DT_F32, torch.bfloat16: MX_DT_BF16}

EXPORTED = ("mx_quantize", "mx_quantize_gather", "mx_quantize_scatter", "mx_dequantize", "mx_transpose", "mx_gemm",
            "mx_gemm_quantize", "mx_gemm_workspace_size", "mx_gemm_noalloc", "mx_gemm_fused_quant_a", "mx_grouped_gemm",
            "mx_grouped_gemm_quantize", "mx_clip_count", "mx_gemm_gated", "mx_gemm_gated_backward",
            "mx_grouped_gemm_gated", "mx_grouped_gemm_gated_backward", "mx_layer_norm", "mx_layer_norm_backward",
            "mx_layer_norm_backward_workspace_size", "mx_dropout", "mx_route", "mx_route_backward", "mx_expert_sort",
            "mx_expert_sort_workspace_size", "mx_expert_dispatch", "mx_expert_combine", "mx_expert_combine_backward",
            "mx_bias_grad", "mx_grouped_bias_grad", "mx_bias_grad_workspace_size", "mx_linear", "mx_linear_backward",
            "mx_grouped_linear", "mx_grouped_linear_backward",
            "mx_last_error", "mx_version")


class MxTensorC(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("K", ctypes.c_int64),
                ("ld_codes", ctypes.c_int64), ("ld_scales", ctypes.c_int64),
                ("block", ctypes.c_int32), ("elem", ctypes.c_int32)]


class QuantCfgC(ctypes.Structure):
    _fields_ = [("axis", ctypes.c_int32), ("block", ctypes.c_int32),
                ("rounding", ctypes.c_int32), ("use_rht", ctypes.c_int32),
                ("rht_sign_mask", ctypes.c_uint32), ("scale_mode", ctypes.c_uint32),
                ("philox_seed", ctypes.c_uint64), ("philox_offset", ctypes.c_uint64)]


class GateCfgC(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("layout", ctypes.c_int32), ("alpha", ctypes.c_float),
                ("limit", ctypes.c_float), ("up_shift", ctypes.c_float)]


class EpilogueCfgC(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("alpha", ctypes.c_float)]


class RouterCfgC(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]


class MXError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"libmxfp4 status {status}: {msg}")
        self.status = status


_lib = None


def load_library(path=LIB_PATH):
    """Load libmxfp4.so and declare its signatures (no GPU is touched)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m mxfp4_microscaling_quantization_mx_amd.build`")
    lib = ctypes.CDLL(path)
    P, I32, I64, U32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32
    PT = ctypes.POINTER(MxTensorC)
    lib.mx_quantize.argtypes = [P, I32, I64, I64, I64, ctypes.POINTER(QuantCfgC), PT, P]
    lib.mx_quantize_gather.argtypes = [P, I32, I64, I64, I64, P, I64, ctypes.POINTER(QuantCfgC), PT, P]
    lib.mx_quantize_scatter.argtypes = [P, I32, I64, I64, I64, P, I32, ctypes.POINTER(QuantCfgC), PT, P]
    lib.mx_dequantize.argtypes = [PT, I32, U32, P, I32, I64, P]
    lib.mx_transpose.argtypes = [PT, PT, P]
    lib.mx_gemm.argtypes = [PT, PT, P, I32, I64, P, ctypes.c_size_t, P]
    lib.mx_gemm_quantize.argtypes = [PT, PT, I32, PT, P]
    lib.mx_gemm_noalloc.argtypes = [PT, PT, P, I32, I64, P]
    lib.mx_gemm_fused_quant_a.argtypes = [P, I32, I64, I64, I64, ctypes.POINTER(QuantCfgC), PT, P, I32, I64, P]
    lib.mx_gemm_workspace_size.argtypes = [I64, I64, I64]
    lib.mx_gemm_workspace_size.restype = ctypes.c_size_t
    lib.mx_grouped_gemm.argtypes = [PT, P, I32, PT, I64, I64, P, I32, I64, P]
    lib.mx_grouped_gemm_quantize.argtypes = [PT, P, I32, PT, I64, I64, I32, PT, P]
    lib.mx_clip_count.argtypes = [P, I32, I64, I64, I64, ctypes.POINTER(QuantCfgC), I32, P, P]
    for f in ("mx_quantize", "mx_quantize_gather", "mx_quantize_scatter", "mx_dequantize", "mx_transpose", "mx_gemm",
              "mx_gemm_quantize", "mx_gemm_noalloc", "mx_gemm_fused_quant_a", "mx_grouped_gemm",
              "mx_grouped_gemm_quantize"):
        getattr(lib, f).restype = ctypes.c_int
    U64, F32, PG = ctypes.c_uint64, ctypes.c_float, ctypes.POINTER(GateCfgC)
    lib.mx_gemm_gated.argtypes = [PT, PT, PG, P, I32, I64, P]
    lib.mx_gemm_gated_backward.argtypes = [PT, PT, PG, P, I32, I64, P, I32, I64, P]
    lib.mx_grouped_gemm_gated.argtypes = [PT, P, I32, PT, I64, I64, PG, P, I32, I64, P]
    lib.mx_grouped_gemm_gated_backward.argtypes = [PT, P, I32, PT, I64, I64, PG, P, I32, I64, P, I32, I64, P]
    lib.mx_layer_norm.argtypes = [P, I32, I64, I64, I64, P, P, I32, F32, P, I64, P, P, P]
    lib.mx_layer_norm_backward.argtypes = [P, P, I32, I64, I64, I64, I64, P, P, P, I32, P, I64, P, P, P,
                                           ctypes.c_size_t, P]
    lib.mx_layer_norm_backward_workspace_size.argtypes = [I64, I64]
    lib.mx_layer_norm_backward_workspace_size.restype = ctypes.c_size_t
    lib.mx_dropout.argtypes = [P, I32, I64, I64, I64, F32, U64, U64, P, I64, P, I64, P]
    for f in ("mx_gemm_gated", "mx_gemm_gated_backward", "mx_grouped_gemm_gated", "mx_grouped_gemm_gated_backward",
              "mx_layer_norm", "mx_layer_norm_backward", "mx_dropout"):
        getattr(lib, f).restype = ctypes.c_int
    SZ, PR = ctypes.c_size_t, ctypes.POINTER(RouterCfgC)
    lib.mx_route.argtypes = [P, I32, I64, I32, I64, I32, PR, P, P, P]
    lib.mx_route_backward.argtypes = [P, P, I32, I64, I32, I64, P, I32, PR, P, I64, P]
    lib.mx_expert_sort.argtypes = [P, I64, I32, I32, P, P, P, P, SZ, P]
    lib.mx_expert_sort_workspace_size.argtypes = [I64, I32, I32]
    lib.mx_expert_sort_workspace_size.restype = SZ
    lib.mx_expert_dispatch.argtypes = [P, I32, I64, I64, I64, P, I32, P, I64, I64, P]
    lib.mx_expert_combine.argtypes = [P, I32, I64, I64, I64, P, P, I64, I32, P, I64, P, I64, P]
    lib.mx_expert_combine_backward.argtypes = [P, I32, I64, I64, I64, P, I64, I64, P, P, I32, P, I64, P, P]
    lib.mx_bias_grad.argtypes = [P, I32, I64, I64, I64, P, I32, P, SZ, P]
    lib.mx_grouped_bias_grad.argtypes = [P, I32, I64, I64, I64, P, I32, P, I32, P, SZ, P]
    lib.mx_bias_grad_workspace_size.argtypes = [I64, I64, I32]
    lib.mx_bias_grad_workspace_size.restype = SZ
    epilogue = [ctypes.POINTER(EpilogueCfgC), P, I32]
    lib.mx_linear.argtypes = [PT, PT, *epilogue, P, I32, I64, P, I32, I64, P]
    lib.mx_grouped_linear.argtypes = [PT, P, I32, PT, I64, I64, *epilogue, I64, P, I32, I64, P, I32, I64, P]
    lib.mx_linear_backward.argtypes = lib.mx_linear.argtypes
    lib.mx_grouped_linear_backward.argtypes = lib.mx_grouped_linear.argtypes
    for f in ("mx_route", "mx_route_backward", "mx_expert_sort", "mx_expert_dispatch", "mx_expert_combine",
              "mx_expert_combine_backward", "mx_bias_grad", "mx_grouped_bias_grad", "mx_linear", "mx_linear_backward",
              "mx_grouped_linear", "mx_grouped_linear_backward"):
        getattr(lib, f).restype = ctypes.c_int
    lib.mx_last_error.restype = ctypes.c_char_p
    lib.mx_last_error.argtypes = []
    lib.mx_version.restype = ctypes.c_char_p
    lib.mx_version.argtypes = []
    _lib = lib
    return lib


def _check(status):
    if status != MX_OK:
        raise MXError(status, _lib.mx_last_error().decode())


def _stream(t, *others):
    """The current stream of t's device, once every tensor of the call (None:
    not given) is known to be there: the library sees addresses only, and a
    host address would fault the GPU."""
    # the handle of torch.cuda.current_stream(t.device), without building the
    # Stream object (2 us of a 4 us launch); a host tensor's index is -1, which
    # would pass for the current device
    d = t.get_device()
    if d < 0:
        raise ValueError("operands must be CUDA tensors")
    for o in others:
        if o is not None and o.get_device() != d:
            raise ValueError("operands must be CUDA tensors on one device")
    return torch._C._cuda_getCurrentRawStream(d)


def _parts(q):
    """The tensors of an MX operand that may be absent."""
    return (q.codes, q.scales) if q is not None else ()


def _ptr(t):
    # an int (None: a null pointer), which the declared argument types convert
    return t.data_ptr() if t is not None else None


@dataclass
class MXTensor:
    """K-major MX operand: codes uint8 [rows, K*bits/8] (MXFP4: K/2), scales
    uint8 [rows, K/32] (1-D) or [rows/32, K/32] (2-D).  Row strides are taken
    from the tensors.  elem: "e2m1" (MXFP4), "e4m3"/"e5m2" (MXFP8) or
    "e2m3"/"e3m2" (MXFP6)."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    K: int
    block: str = "1d"
    elem: str = "e2m1"

    def c_struct(self):
        elem, bits = _ELEM[self.elem]
        codes, scales = self.codes.stride(), self.scales.stride()
        return MxTensorC(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.K,
                         codes[0] if len(codes) == 2 else self.K * bits // 8,
                         scales[0] if len(scales) == 2 else self.K // 32, _BLOCK[self.block], elem)


def empty_mx(rows, K, block="1d", device="cuda", experts=None, elem="e2m1"):
    """Allocate an uninitialised MX operand (codes + scales) on `device`.

    Code rows are padded to a multiple of 128 bytes and scale rows to a
    multiple of 16 bytes (the row strides are carried in the tensors), so the
    GEMMs' row segments start on cache-line boundaries and their scale fetches
    are aligned.  With `experts=E` the tensors get a leading expert dimension
    (the stacked weights of grouped_gemm); expert e is `expert(q, e)`."""
    srows = rows // 32 if block == "2d" else rows
    lead = () if experts is None else (experts,)
    cb = K * _ELEM[elem][1] // 8
    ldc = (cb + 127) // 128 * 128
    codes = torch.empty(lead + (rows, ldc), dtype=torch.uint8, device=device)[..., :cb]
    ld = (K // 32 + 15) // 16 * 16
    scales = torch.empty(lead + (srows, ld), dtype=torch.uint8, device=device)[..., :K // 32]
    return MXTensor(codes, scales, rows, K, block, elem)


def expert(q, e):
    """View of expert e of a stacked operand from empty_mx(..., experts=E)."""
    return MXTensor(q.codes[e], q.scales[e], q.rows, q.K, q.block, q.elem)


def quantize(x, axis="last", block="1d", rounding="rne", rht_mask=None, seed=0, offset=0,
             out=None, scale_mode="floor", elem="e2m1"):
    """Quantize a 2-D bf16/fp32 CUDA tensor to MXFP4 (or, with elem, MXFP8 /
    MXFP6; see mx_quantize in include/mx.h).

    axis="dim0" blocks along dim 0 and returns the quantized transpose.
    scale_mode: "floor" (the reference rule), "round_up" or "prescale_3_4".
    With `out` given, its element type is the one produced."""
    lib = load_library()
    if x.dim() != 2 or x.dtype not in _DTYPE or not x.is_cuda:
        raise ValueError("quantize expects a 2-D bf16/float32 CUDA tensor")
    if x.stride(1) != 1:
        raise ValueError("quantize expects a row-major tensor (stride(1) == 1)")
    st = _stream(x, *_parts(out))
    R, C = x.shape
    rows, K = (C, R) if axis == "dim0" else (R, C)
    if out is None:
        out = empty_mx(rows, K, block, x.device, elem=elem)
    cfg = QuantCfgC(_AXIS[axis], _BLOCK[block], _ROUND[rounding], int(rht_mask is not None),
                    (rht_mask or 0) & 0xFFFFFFFF, _SCALE[scale_mode], seed & (2**64 - 1),
                    offset & (2**64 - 1))
    ot = out.c_struct()
    _check(lib.mx_quantize(_ptr(x), _DTYPE[x.dtype], R, C, x.stride(0), ctypes.byref(cfg),
                           ctypes.byref(ot), st))
    return out


def clip_count(x, axis="last", block="1d", rht_mask=None, scale_mode="floor", elem="e2m1", out=None):
    """Clipping statistic of quantizing x with these settings: the number of
    elements that saturate at the element type's largest normal (see
    mx_clip_count in include/mx.h).  Returns a one-element int64 CUDA tensor;
    with `out` given (one int64 element), the count is added to it."""
    lib = load_library()
    if x.dim() != 2 or x.dtype not in _DTYPE or not x.is_cuda:
        raise ValueError("clip_count expects a 2-D bf16/float32 CUDA tensor")
    if x.stride(1) != 1:
        raise ValueError("clip_count expects a row-major tensor (stride(1) == 1)")
    st = _stream(x, out)
    if out is None:
        out = torch.zeros(1, dtype=torch.int64, device=x.device)
    elif out.dtype != torch.int64 or out.numel() != 1 or not out.is_cuda:
        raise ValueError("clip_count: out must be a one-element int64 CUDA tensor")
    R, C = x.shape
    cfg = QuantCfgC(_AXIS[axis], _BLOCK[block], _ROUND["rne"], int(rht_mask is not None),
                    (rht_mask or 0) & 0xFFFFFFFF, _SCALE[scale_mode], 0, 0)
    _check(lib.mx_clip_count(_ptr(x), _DTYPE[x.dtype], R, C, x.stride(0), ctypes.byref(cfg), _ELEM[elem][0],
                             _ptr(out), st))
    return out


def quantize_gather(x, rows, rounding="rne", rht_mask=None, seed=0, offset=0, out=None, scale_mode="floor"):
    """Quantize the rows x[rows[i]] of a 2-D bf16/fp32 CUDA tensor, 1-D blocks
    along the last dim (see mx_quantize_gather in include/mx.h).  `rows` is an
    int32 CUDA tensor; indices outside [0, x.shape[0]) give NaN blocks."""
    lib = load_library()
    if x.dim() != 2 or x.dtype not in _DTYPE or not x.is_cuda:
        raise ValueError("quantize_gather expects a 2-D bf16/float32 CUDA tensor")
    if x.stride(1) != 1:
        raise ValueError("quantize_gather expects a row-major tensor (stride(1) == 1)")
    if rows.dtype != torch.int32 or rows.dim() != 1 or not rows.is_cuda or not rows.is_contiguous():
        raise ValueError("quantize_gather expects rows as a contiguous 1-D int32 CUDA tensor")
    st = _stream(x, rows, *_parts(out))
    R, C = x.shape
    n = rows.shape[0]
    if out is None:
        out = empty_mx(n, C, "1d", x.device)
    cfg = QuantCfgC(_AXIS["last"], _BLOCK["1d"], _ROUND[rounding], int(rht_mask is not None),
                    (rht_mask or 0) & 0xFFFFFFFF, _SCALE[scale_mode], seed & (2**64 - 1),
                    offset & (2**64 - 1))
    ot = out.c_struct()
    _check(lib.mx_quantize_gather(_ptr(x), _DTYPE[x.dtype], R, C, x.stride(0), _ptr(rows), n,
                                  ctypes.byref(cfg), ctypes.byref(ot), st))
    return out


def quantize_scatter(x, dest, k, rows_out=None, rht_mask=None, out=None, scale_mode="floor"):
    """Quantize each row of a 2-D bf16/fp32 CUDA tensor once (1-D blocks along
    the last dim, RNE) and store it to its k destination rows dest[t*k + j]
    (see mx_quantize_scatter).  `dest` is an int32 CUDA tensor of x.shape[0]*k
    entries; out (or a new [rows_out, C] operand) receives the rows."""
    lib = load_library()
    if x.dim() != 2 or x.dtype not in _DTYPE or not x.is_cuda:
        raise ValueError("quantize_scatter expects a 2-D bf16/float32 CUDA tensor")
    if x.stride(1) != 1:
        raise ValueError("quantize_scatter expects a row-major tensor (stride(1) == 1)")
    st = _stream(x, dest, *_parts(out))
    R, C = x.shape
    if dest.dtype != torch.int32 or not dest.is_cuda or not dest.is_contiguous() or dest.numel() != R * k:
        raise ValueError("quantize_scatter expects dest as a contiguous int32 CUDA tensor of R*k entries")
    if out is None:
        out = empty_mx(R * k if rows_out is None else rows_out, C, "1d", x.device)
    cfg = QuantCfgC(_AXIS["last"], _BLOCK["1d"], _ROUND["rne"], int(rht_mask is not None),
                    (rht_mask or 0) & 0xFFFFFFFF, _SCALE[scale_mode], 0, 0)
    ot = out.c_struct()
    _check(lib.mx_quantize_scatter(_ptr(x), _DTYPE[x.dtype], R, C, x.stride(0), _ptr(dest), k,
                                   ctypes.byref(cfg), ctypes.byref(ot), st))
    return out


def dequantize(q, dtype=torch.float32, inverse_rht_mask=None, out=None):
    """Decode an MX operand to a [rows, K] tensor (see mx_dequantize)."""
    lib = load_library()
    st = _stream(q.codes, q.scales, out)
    if out is None:
        out = torch.empty((q.rows, q.K), dtype=dtype, device=q.codes.device)
    qt = q.c_struct()
    _check(lib.mx_dequantize(ctypes.byref(qt), int(inverse_rht_mask is not None),
                             (inverse_rht_mask or 0) & 0xFFFFFFFF, _ptr(out), _DTYPE[out.dtype],
                             out.stride(0), st))
    return out


def transpose(q, out=None):
    """Exact transpose of an operand with 2-D (32x32) blocks: [R, C] -> [C, R]
    (see mx_transpose)."""
    lib = load_library()
    st = _stream(q.codes, q.scales, *_parts(out))
    if out is None:
        out = empty_mx(q.K, q.rows, "2d", device=q.codes.device, elem=q.elem)
    it, ot = q.c_struct(), out.c_struct()
    _check(lib.mx_transpose(ctypes.byref(it), ctypes.byref(ot), st))
    return out


_WORKSPACES = {}


def gemm_workspace(M, N, K, device="cuda"):
    """A workspace for mx_gemm of an M x N x K problem (None if it needs none):
    one zero-filled buffer per device, grown on demand and reused (every call
    leaves it fit for the next, see mx_gemm_workspace_size).  Calls that share
    it must not overlap, so callers on several streams pass their own."""
    n = load_library().mx_gemm_workspace_size(M, N, K)
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError("gemm_workspace: the workspace is a CUDA tensor")
    if not n:
        return None
    key = dev.index if dev.index is not None else torch.cuda.current_device()
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < n:
        ws = torch.zeros(n, dtype=torch.uint8, device=dev)
        _WORKSPACES[key] = ws
    return ws


def gemm(a, b, out_dtype=torch.float32, out=None, workspace=None):
    """C = A * B^T for MX operands A [M, K], B [N, K] (see mx_gemm).  Shapes
    that mx_gemm splits along K use `workspace` (a zero-filled uint8 CUDA
    tensor of at least mx_gemm_workspace_size bytes) or the per-device one of
    gemm_workspace."""
    lib = load_library()
    st = _stream(a.codes, a.scales, b.codes, b.scales, out, workspace)
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=out_dtype, device=a.codes.device)
    ws = lib.mx_gemm_workspace_size(a.rows, b.rows, a.K)
    if ws and workspace is None:
        workspace = gemm_workspace(a.rows, b.rows, a.K, a.codes.device)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    at, bt = a.c_struct(), b.c_struct()
    _check(lib.mx_gemm(ctypes.byref(at), ctypes.byref(bt), _ptr(out), _DTYPE[out.dtype],
                       out.stride(0), _ptr(workspace), nbytes, st))
    return out


def gemm_noalloc(a, b, out_dtype=torch.float32, out=None):
    """C = A * B^T through mx_gemm_noalloc: the library's own split-K scratch,
    no workspace argument (for callers that cannot allocate; the output is
    still the caller's)."""
    lib = load_library()
    st = _stream(a.codes, a.scales, b.codes, b.scales, out)
    if out is None:
        out = torch.empty((a.rows, b.rows), dtype=out_dtype, device=a.codes.device)
    at, bt = a.c_struct(), b.c_struct()
    _check(lib.mx_gemm_noalloc(ctypes.byref(at), ctypes.byref(bt), _ptr(out), _DTYPE[out.dtype], out.stride(0),
                               st))
    return out


def gemm_fused_quant_a(a, b, out_dtype=torch.float32, out=None, rht_mask=None, scale_mode="floor"):
    """C = Q(A) * B^T with A a 2-D bf16 CUDA tensor [M, K] quantized to MXFP4
    inside the GEMM's operand load (RNE, 1-D blocks along K, optional
    transform; see mx_gemm_fused_quant_a) and B an MXFP4 operand [N, K]."""
    lib = load_library()
    if a.dim() != 2 or a.dtype not in _DTYPE or not a.is_cuda or a.stride(1) != 1:
        raise ValueError("gemm_fused_quant_a expects a row-major 2-D bf16 CUDA tensor")
    st = _stream(a, b.codes, b.scales, out)
    M, K = a.shape
    if out is None:
        out = torch.empty((M, b.rows), dtype=out_dtype, device=a.device)
    cfg = QuantCfgC(_AXIS["last"], _BLOCK["1d"], _ROUND["rne"], int(rht_mask is not None),
                    (rht_mask or 0) & 0xFFFFFFFF, _SCALE[scale_mode], 0, 0)
    bt = b.c_struct()
    _check(lib.mx_gemm_fused_quant_a(_ptr(a), _DTYPE[a.dtype], M, K, a.stride(0), ctypes.byref(cfg), ctypes.byref(bt),
                                     _ptr(out), _DTYPE[out.dtype], out.stride(0), st))
    return out


def gemm_quantize(a, b, scale_mode="floor", out=None):
    """A * B^T quantized along N into an MXFP4 operand [M, N] (1-D blocks, RNE)
    in the GEMM epilogue (see mx_gemm_quantize)."""
    lib = load_library()
    st = _stream(a.codes, a.scales, b.codes, b.scales, *_parts(out))
    if out is None:
        out = empty_mx(a.rows, b.rows, device=a.codes.device)
    at, bt, ot = a.c_struct(), b.c_struct(), out.c_struct()
    _check(lib.mx_gemm_quantize(ctypes.byref(at), ctypes.byref(bt), _SCALE[scale_mode], ctypes.byref(ot),
                                st))
    return out


def _check_offsets(offsets, E):
    if (offsets.dtype != torch.int32 or not offsets.is_cuda or offsets.numel() != E + 1
            or not offsets.is_contiguous()):
        raise ValueError("offsets must be a contiguous int32 CUDA tensor of E+1 entries")


def grouped_gemm(a, offsets, b, out_dtype=torch.bfloat16, out=None):
    """MoE grouped GEMM (see mx_grouped_gemm).

    a: MXTensor [M, K] with rows grouped by expert; offsets: int32 CUDA tensor
    [E+1]; b: MXTensor whose codes are [E, N, K/2] and scales [E, N/32, K/32]
    (2-D) or [E, N, K/32] (1-D)."""
    lib = load_library()
    E = b.codes.shape[0]
    _check_offsets(offsets, E)
    st = _stream(a.codes, a.scales, b.codes, b.scales, offsets, out)
    N = b.codes.shape[1]
    if out is None:
        out = torch.empty((a.rows, N), dtype=out_dtype, device=a.codes.device)
    b0 = MxTensorC(b.codes.data_ptr(), b.scales.data_ptr(), N, b.K, b.codes.stride(1),
                   b.scales.stride(1), _BLOCK[b.block], _ELEM[b.elem][0])
    at = a.c_struct()
    _check(lib.mx_grouped_gemm(ctypes.byref(at), _ptr(offsets), E, ctypes.byref(b0),
                               b.codes.stride(0), b.scales.stride(0), _ptr(out),
                               _DTYPE[out.dtype], out.stride(0), st))
    return out


def grouped_gemm_quantize(a, offsets, b, scale_mode="floor", out=None):
    """The grouped product quantized along N into an MXFP4 operand [M, N] in
    the GEMM epilogue (see mx_grouped_gemm_quantize); arguments as
    grouped_gemm."""
    lib = load_library()
    E = b.codes.shape[0]
    _check_offsets(offsets, E)
    st = _stream(a.codes, a.scales, b.codes, b.scales, offsets, *_parts(out))
    N = b.codes.shape[1]
    if out is None:
        out = empty_mx(a.rows, N, device=a.codes.device)
    b0 = MxTensorC(b.codes.data_ptr(), b.scales.data_ptr(), N, b.K, b.codes.stride(1),
                   b.scales.stride(1), _BLOCK[b.block], _ELEM[b.elem][0])
    at, ot = a.c_struct(), out.c_struct()
    _check(lib.mx_grouped_gemm_quantize(ctypes.byref(at), _ptr(offsets), E, ctypes.byref(b0), b.codes.stride(0),
                                        b.scales.stride(0), _SCALE[scale_mode], ctypes.byref(ot),
                                        st))
    return out


@dataclass(frozen=True)
class Gate:
    """A gated block: act(min(g, limit)) * (clamp(u, -limit, limit) + up_shift)
    for the gate and up projections g, u (mx_gate_cfg in include/mx.h).  act:
    "silu" (g * sigmoid(alpha g)), "gelu" or "gelu_tanh" (which have no alpha
    and ignore it); limit None: no clamp.  layout: gate and up rows of the
    weight "interleaved" or in two "halves" (gates first)."""
    act: str = "silu"
    alpha: float = 1.0
    limit: float = None
    up_shift: float = 0.0
    layout: str = "interleaved"

    def __post_init__(self):
        # the library's 0 is no clamp
        if self.limit is not None and ctypes.c_float(self.limit).value == 0.0:
            raise ValueError("Gate: a limit of 0 cannot be expressed (None: no clamp)")

    def c_struct(self):
        return GateCfgC(_ACT[self.act], _GATE_LAYOUT[self.layout], self.alpha,
                        0.0 if self.limit is None else self.limit, self.up_shift)


def _check_rows(t, what, shape=None, dtype=None):
    """The row stride of a row-major matrix (where it is: _stream).  One row's
    stride means nothing and may be anything."""
    st = t.stride()
    if len(st) != 2 or t.dtype not in _DTYPE:
        raise ValueError(f"{what} must be a 2-D bf16/float32 CUDA tensor")
    R, C = t.shape
    if st[1] != 1 and C > 1:
        raise ValueError(f"{what} must be row-major (stride(1) == 1)")
    if shape is not None and (R, C) != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}")
    return st[0] if R > 1 else C


def _gated(what, a, b, gate, out, out_dtype, dh, offsets):
    lib = load_library()
    st = _stream(a.codes, a.scales, b.codes, b.scales, offsets, dh, out)
    backward = dh is not None
    if offsets is not None:
        E, rows = b.codes.shape[0], b.codes.shape[1]
        _check_offsets(offsets, E)
        bt = MxTensorC(b.codes.data_ptr(), b.scales.data_ptr(), rows, b.K, b.codes.stride(1), b.scales.stride(1),
                       _BLOCK[b.block], _ELEM[b.elem][0])
        group = (_ptr(offsets), E, ctypes.byref(bt), b.codes.stride(0), b.scales.stride(0))
    else:
        rows, bt = b.rows, b.c_struct()
        group = (ctypes.byref(bt),)
    N = rows // 2
    shape = (a.rows, rows if backward else N)
    if out is None:
        out, ldo = a.codes.new_empty(shape, dtype=out_dtype), shape[1]
    else:
        ldo = _check_rows(out, f"{what}: out", shape)
    args = ()
    if backward:
        ldh = _check_rows(dh, f"{what}: dh", (a.rows, N))
        args = (_ptr(dh), _DTYPE[dh.dtype], ldh)
    at, gc = a.c_struct(), gate.c_struct()
    _check(getattr(lib, what)(ctypes.byref(at), *group, ctypes.byref(gc), *args, _ptr(out), _DTYPE[out.dtype],
                              ldo, st))
    return out


def gemm_gated(a, b, gate=Gate(), out_dtype=torch.bfloat16, out=None):
    """The gated feed-forward block of MX operands a [M, K] and b [2N, K]
    (gate and up rows): both projections, the activation and the product in
    one kernel, [M, N] (see mx_gemm_gated)."""
    return _gated("mx_gemm_gated", a, b, gate, out, out_dtype, None, None)


def gemm_gated_backward(a, b, dh, gate=Gate(), out_dtype=torch.bfloat16, out=None):
    """The gradient [M, 2N] of gemm_gated's projections for the gradient dh
    [M, N] of its output, the projections recomputed from a and b (see
    mx_gemm_gated_backward); its columns are in the order of b's rows."""
    return _gated("mx_gemm_gated_backward", a, b, gate, out, out_dtype, dh, None)


def grouped_gemm_gated(a, offsets, b, gate=Gate(), out_dtype=torch.bfloat16, out=None):
    """gemm_gated for rows grouped by expert; a, offsets and the stacked b
    [E, 2N, K] as in grouped_gemm (see mx_grouped_gemm_gated).  Rows past
    offsets[E] of the output are not written."""
    return _gated("mx_grouped_gemm_gated", a, b, gate, out, out_dtype, None, offsets)


def grouped_gemm_gated_backward(a, offsets, b, dh, gate=Gate(), out_dtype=torch.bfloat16, out=None):
    """gemm_gated_backward for rows grouped by expert."""
    return _gated("mx_grouped_gemm_gated_backward", a, b, gate, out, out_dtype, dh, offsets)


def _norm_param(t, C, dtype, what):
    if t.shape != (C,) or t.dtype not in _DTYPE or not t.is_cuda or (t.stride(0) != 1 and C > 1):
        raise ValueError(f"{what} must be a contiguous bf16/float32 CUDA tensor of {C} entries")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must have the weight's dtype")


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None):
    """Layer norm of the rows of a 2-D bf16/float32 CUDA tensor (see
    mx_layer_norm): (y, mean, rstd), the row statistics in float32 for
    layer_norm_backward."""
    lib = load_library()
    ldx = _check_rows(x, "layer_norm: x")
    st = _stream(x, weight, bias, out)
    R, C = x.shape
    if weight is not None:
        _norm_param(weight, C, None, "layer_norm: weight")
    if bias is not None:
        _norm_param(bias, C, None if weight is None else weight.dtype, "layer_norm: bias")
    if out is None:
        out, ldo = x.new_empty((R, C)), C
    else:
        ldo = _check_rows(out, "layer_norm: out", (R, C), x.dtype)
    mean, rstd = x.new_empty(R, dtype=torch.float32), x.new_empty(R, dtype=torch.float32)
    if not C:                                   # (the library writes nothing then)
        mean.fill_(float("nan"))
        rstd.fill_(float("nan"))
    wd = weight if weight is not None else bias
    _check(lib.mx_layer_norm(_ptr(x), _DTYPE[x.dtype], R, C, ldx, _ptr(weight), _ptr(bias),
                             MX_DT_F32 if wd is None else _DTYPE[wd.dtype], eps, _ptr(out), ldo,
                             _ptr(mean), _ptr(rstd), st))
    return out, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, out=None, param_dtype=None):
    """The gradients (dx, dweight, dbias) of layer_norm (see
    mx_layer_norm_backward).  dweight and dbias have the weight's dtype, or
    param_dtype without one (default float32); out receives dx."""
    lib = load_library()
    ldx = _check_rows(x, "layer_norm_backward: x")
    R, C = x.shape
    lddy = _check_rows(dy, "layer_norm_backward: dy", (R, C), x.dtype)
    st = _stream(x, dy, mean, rstd, weight, out)
    for t, n in ((mean, "mean"), (rstd, "rstd")):
        if t.shape != (R,) or t.dtype != torch.float32 or not t.is_cuda or (R > 1 and t.stride(0) != 1):
            raise ValueError(f"layer_norm_backward: {n} must be a contiguous float32 CUDA tensor of {R} entries")
    if weight is not None:
        _norm_param(weight, C, param_dtype, "layer_norm_backward: weight")
        param_dtype = weight.dtype
    elif param_dtype is None:
        param_dtype = torch.float32
    if out is None:
        out, lddx = x.new_empty((R, C)), C
    else:
        lddx = _check_rows(out, "layer_norm_backward: out", (R, C), x.dtype)
    dweight, dbias = x.new_empty(C, dtype=param_dtype), x.new_empty(C, dtype=param_dtype)
    nbytes = lib.mx_layer_norm_backward_workspace_size(R, C)
    ws = x.new_empty(nbytes, dtype=torch.uint8)
    _check(lib.mx_layer_norm_backward(_ptr(dy), _ptr(x), _DTYPE[x.dtype], R, C, lddy, ldx, _ptr(mean),
                                      _ptr(rstd), _ptr(weight), _DTYPE[param_dtype], _ptr(out), lddx,
                                      _ptr(dweight), _ptr(dbias), _ptr(ws), nbytes, st))
    return out, dweight, dbias


def dropout(x, p, seed=0, offset=0, residual=None, out=None):
    """Dropout of a 2-D bf16/float32 CUDA tensor from Philox draws, plus an
    optional residual (see mx_dropout).  The backward pass is this call on the
    gradient with the same p, seed and offset and no residual."""
    lib = load_library()
    ldx = _check_rows(x, "dropout: x")
    st = _stream(x, residual, out)
    R, C = x.shape
    ldr = 0
    if residual is not None:
        ldr = _check_rows(residual, "dropout: residual", (R, C), x.dtype)
    if out is None:
        out, ldo = x.new_empty((R, C)), C
    else:
        ldo = _check_rows(out, "dropout: out", (R, C), x.dtype)
    _check(lib.mx_dropout(_ptr(x), _DTYPE[x.dtype], R, C, ldx, p, seed & (2**64 - 1), offset & (2**64 - 1),
                          _ptr(residual), ldr, _ptr(out), ldo, st))
    return out


@dataclass(frozen=True)
class Router:
    """How routing weights come from logits (mx_router_cfg in include/mx.h).
    score: "softmax" or "sigmoid"; renormalize: the chosen scores of a token are
    divided by their sum; scale: a factor of every weight."""
    score: str = "softmax"
    renormalize: bool = True
    scale: float = 1.0

    @functools.cached_property
    def _cfg(self):                             # (the library only reads it)
        return RouterCfgC(_SCORE[self.score], int(self.renormalize), self.scale)

    def c_struct(self):
        return self._cfg


@functools.lru_cache(maxsize=64)
def _epilogue_cfg(act, alpha):
    return EpilogueCfgC(_EPILOGUE_ACT[act], alpha)


# (sizes alone decide these: asked once per shape)
@functools.lru_cache(maxsize=256)
def _sort_workspace(T, top, E):
    return load_library().mx_expert_sort_workspace_size(T, top, E)


@functools.lru_cache(maxsize=256)
def _bias_grad_workspace(M, N, E):
    return load_library().mx_bias_grad_workspace_size(M, N, E)


def _slots(t, what, dtype, shape=None):
    """Check a contiguous [T, top] array of slots (where it is: _stream)."""
    if t.dim() != 2 or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous 2-D {dtype} CUDA tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}")


def _size(n, most):
    """A size as the library is told it, and as its outputs are allocated: the library
    turns down what is outside [0, most] before it looks at a buffer, so such a size
    allocates no more than that."""
    return max(-1, min(n, most + 1)), max(0, min(n, most))


def route(logits, top, router=Router()):
    """The `top` experts of every token and their weights from the logits
    [T, E], bf16 or float32 (see mx_route): (ids int32 [T, top], weights
    float32 [T, top])."""
    lib = load_library()
    ld = _check_rows(logits, "route: logits")
    st = _stream(logits)
    T, E = logits.shape
    top, n = _size(top, _CHOICES_MAX)
    ids = logits.new_empty((T, n), dtype=torch.int32)
    weights = logits.new_empty((T, n), dtype=torch.float32)
    cfg = router.c_struct()
    _check(lib.mx_route(_ptr(logits), _DTYPE[logits.dtype], T, E, ld, top, ctypes.byref(cfg), _ptr(ids),
                        _ptr(weights), st))
    return ids, weights


def route_backward(dweights, logits, ids, router=Router(), out=None):
    """The gradient [T, E] of route's weights by the logits for the gradient
    dweights [T, top] and the choice ids (see mx_route_backward)."""
    lib = load_library()
    ld = _check_rows(logits, "route_backward: logits")
    T, E = logits.shape
    _slots(ids, "route_backward: ids", torch.int32)
    _slots(dweights, "route_backward: dweights", torch.float32, ids.shape)
    if ids.shape[0] != T:
        raise ValueError(f"route_backward: ids must have {T} rows")
    st = _stream(logits, dweights, ids, out)
    if out is None:
        out, ldo = logits.new_empty((T, E)), E
    else:
        ldo = _check_rows(out, "route_backward: out", (T, E), logits.dtype)
    cfg = router.c_struct()
    _check(lib.mx_route_backward(_ptr(dweights), _ptr(logits), _DTYPE[logits.dtype], T, E, ld, _ptr(ids),
                                 ids.shape[1], ctypes.byref(cfg), _ptr(out), ldo, st))
    return out


def expert_sort(ids, E):
    """The slots (token, choice) of ids [T, top] int32 sorted by expert (see
    mx_expert_sort): (offsets [E+1], rows [T*top], dest [T, top]), int32.
    offsets is what the grouped products take, rows what quantize_gather does
    and dest what quantize_scatter, expert_dispatch and expert_combine do; a
    slot whose id is outside [0, E) is dropped (dest -1)."""
    lib = load_library()
    _slots(ids, "expert_sort: ids", torch.int32)
    st = _stream(ids)
    T, top = ids.shape
    E, n = _size(E, _EXPERTS_MAX)
    offsets, rows, dest = ids.new_empty(n + 1), ids.new_empty(T * top), ids.new_empty((T, top))
    nbytes = _sort_workspace(T, top, E)
    ws = ids.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
    _check(lib.mx_expert_sort(_ptr(ids), T, top, E, _ptr(offsets), _ptr(rows), _ptr(dest), _ptr(ws), nbytes, st))
    return offsets, rows, dest


def expert_dispatch(x, dest, rows_out=None, out=None):
    """Rows x[t] of a 2-D bf16/float32 CUDA tensor copied to their sorted rows
    dest[t, j] (see mx_expert_dispatch); out (or a new [rows_out, C] tensor, by
    default a row per slot) receives them.  Rows that dest does not name are not
    written.  The gradient is expert_combine without weights."""
    lib = load_library()
    ldx = _check_rows(x, "expert_dispatch: x")
    T, C = x.shape
    _slots(dest, "expert_dispatch: dest", torch.int32)
    if dest.shape[0] != T:
        raise ValueError(f"expert_dispatch: dest must have {T} rows")
    st = _stream(x, dest, out)
    if out is None:
        rows_out = dest.numel() if rows_out is None else rows_out
        out, ldo = x.new_empty((rows_out, C)), C
    else:
        ldo = _check_rows(out, "expert_dispatch: out", (out.shape[0] if rows_out is None else rows_out, C), x.dtype)
    _check(lib.mx_expert_dispatch(_ptr(x), _DTYPE[x.dtype], T, C, ldx, _ptr(dest), dest.shape[1], _ptr(out),
                                  out.shape[0], ldo, st))
    return out


def expert_combine(y, dest, weights=None, residual=None, out=None):
    """The expert rows y [rows, C] back to their tokens (see mx_expert_combine):
    out[t] = sum_j weights[t, j] * y[dest[t, j]] + residual[t], weights float32
    [T, top] (None: 1).  Dropped slots add nothing; out may be residual."""
    lib = load_library()
    ldy = _check_rows(y, "expert_combine: y")
    rows, C = y.shape
    _slots(dest, "expert_combine: dest", torch.int32)
    T, top = dest.shape
    if weights is not None:
        _slots(weights, "expert_combine: weights", torch.float32, dest.shape)
    ldr = 0
    if residual is not None:
        ldr = _check_rows(residual, "expert_combine: residual", (T, C), y.dtype)
    st = _stream(y, dest, weights, residual, out)
    if out is None:
        out, ldo = y.new_empty((T, C)), C
    else:
        ldo = _check_rows(out, "expert_combine: out", (T, C), y.dtype)
    _check(lib.mx_expert_combine(_ptr(y), _DTYPE[y.dtype], rows, C, ldy, _ptr(dest), _ptr(weights), T, top,
                                 _ptr(residual), ldr, _ptr(out), ldo, st))
    return out


def expert_combine_backward(dout, y, dest, weights, out=None):
    """The gradients (dy, dweights) of expert_combine for the gradient dout
    [T, C] (see mx_expert_combine_backward); out receives dy [rows, C], whose
    rows that dest does not name are not written."""
    lib = load_library()
    ldy = _check_rows(y, "expert_combine_backward: y")
    rows, C = y.shape
    _slots(dest, "expert_combine_backward: dest", torch.int32)
    _slots(weights, "expert_combine_backward: weights", torch.float32, dest.shape)
    T, top = dest.shape
    lddo = _check_rows(dout, "expert_combine_backward: dout", (T, C), y.dtype)
    st = _stream(y, dout, dest, weights, out)
    if out is None:
        out, ldo = y.new_empty((rows, C)), C
    else:
        ldo = _check_rows(out, "expert_combine_backward: out", (rows, C), y.dtype)
    dweights = weights.new_empty((T, top))
    _check(lib.mx_expert_combine_backward(_ptr(dout), _DTYPE[y.dtype], T, C, lddo, _ptr(y), rows, ldy, _ptr(dest),
                                          _ptr(weights), top, _ptr(out), ldo, _ptr(dweights), st))
    return out, dweights


def _linear(what, a, b, offsets, bias, act, alpha, r, r_name, out_dtype, out):
    lib = load_library()
    st = _stream(a.codes, a.scales, b.codes, b.scales, offsets, bias, r, out)
    if offsets is not None:
        E, N = b.codes.shape[0], b.codes.shape[1]
        _check_offsets(offsets, E)
        bt = MxTensorC(b.codes.data_ptr(), b.scales.data_ptr(), N, b.K, b.codes.stride(1), b.scales.stride(1),
                       _BLOCK[b.block], _ELEM[b.elem][0])
        group = (_ptr(offsets), E, ctypes.byref(bt), b.codes.stride(0), b.scales.stride(0))
    else:
        N, bt = b.rows, b.c_struct()
        group = (ctypes.byref(bt),)
    epilogue = (None, MX_DT_F32)
    if bias is not None:
        if offsets is None:
            _norm_param(bias, N, None, f"{what}: bias")
            stride = ()
        else:
            stride = (_check_rows(bias, f"{what}: bias", (E, N)),)
        epilogue = (_ptr(bias), _DTYPE[bias.dtype], *stride)
    elif offsets is not None:
        epilogue += (0,)
    shape = (a.rows, N)
    ldr, rd = 0, MX_DT_F32
    if r is not None:
        ldr, rd = _check_rows(r, f"{what}: {r_name}", shape), _DTYPE[r.dtype]
    if out is None:
        out, ldo = a.codes.new_empty(shape, dtype=out_dtype), N
    else:
        ldo = _check_rows(out, f"{what}: out", shape)
    at, cfg = a.c_struct(), _epilogue_cfg(act, alpha)
    _check(getattr(lib, what)(ctypes.byref(at), *group, ctypes.byref(cfg), *epilogue, _ptr(r), rd, ldr, _ptr(out),
                              _DTYPE[out.dtype], ldo, st))
    return out


def linear(a, b, bias=None, act=None, residual=None, alpha=1.0, out_dtype=torch.bfloat16, out=None):
    """act(A B^T + bias) + residual for MX operands a [M, K] and b [N, K], the
    bias [N], activation (None, "silu" with slope alpha, "gelu", "gelu_tanh")
    and residual [M, N] in the product's epilogue (see mx_linear).  bias and
    residual may be bf16 or float32; out may be residual."""
    return _linear("mx_linear", a, b, None, bias, act, alpha, residual, "residual", out_dtype, out)


def linear_backward(a, b, dy, bias=None, act="gelu", alpha=1.0, out_dtype=torch.bfloat16, out=None):
    """The gradient dy * act'(A B^T + bias) [M, N] of linear through its
    activation, the product recomputed from a and b (see mx_linear_backward);
    the bias's gradient is bias_grad of it."""
    return _linear("mx_linear_backward", a, b, None, bias, act, alpha, dy, "dy", out_dtype, out)


def grouped_linear(a, offsets, b, bias=None, act=None, residual=None, alpha=1.0, out_dtype=torch.bfloat16, out=None):
    """linear for rows grouped by expert; a, offsets and the stacked b [E, N, K]
    as in grouped_gemm, bias [E, N] (see mx_grouped_linear).  Rows past
    offsets[E] of the output are not written."""
    return _linear("mx_grouped_linear", a, b, offsets, bias, act, alpha, residual, "residual", out_dtype, out)


def grouped_linear_backward(a, offsets, b, dy, bias=None, act="gelu", alpha=1.0, out_dtype=torch.bfloat16, out=None):
    """linear_backward for rows grouped by expert."""
    return _linear("mx_grouped_linear_backward", a, b, offsets, bias, act, alpha, dy, "dy", out_dtype, out)


def bias_grad(dp, offsets=None, dtype=torch.float32):
    """The sums of the columns of dp [M, N], the gradient of a bias [N]; with
    offsets [E+1] those of each expert's rows, [E, N] (see mx_bias_grad and
    mx_grouped_bias_grad)."""
    lib = load_library()
    ld = _check_rows(dp, "bias_grad: dp")
    if dtype not in _DTYPE:
        raise ValueError("bias_grad: dtype must be bf16 or float32")
    M, N = dp.shape
    st = _stream(dp, offsets)
    if offsets is None:
        E, group, shape, f = 1, (), (N,), lib.mx_bias_grad
    else:
        E = offsets.numel() - 1
        _check_offsets(offsets, E)
        if E < 1:
            raise ValueError("bias_grad: offsets must have at least two entries")
        group, shape, f = (_ptr(offsets), E), (E, N), lib.mx_grouped_bias_grad
    out = dp.new_empty(shape) if dtype == dp.dtype else dp.new_empty(shape, dtype=dtype)
    nbytes = _bias_grad_workspace(M, N, E)
    ws = dp.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
    _check(f(_ptr(dp), _DTYPE[dp.dtype], M, N, ld, *group, _ptr(out), _DTYPE[dtype], _ptr(ws), nbytes, st))
    return out


def version():
    return load_library().mx_version().decode()
