"""Refusals of the linear layer's entry points: every call here is turned down (or is
a no-op) on the host, before anything is launched."""
import ctypes
import os

import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx
from test_binding_devices_experts import StubLibrary, on

P, B = ctypes.c_void_p, ctypes.byref
BAD, UNSUP, OK = mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED, mx.MX_OK
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mx.LIB_PATH):
        pytest.skip("libmxfp4.so not built")
    return mx.load_library()


def _tensor(rows, K, block=0, codes=16, scales=16, ldc=None, elem=0):
    return mx.MxTensorC(codes, scales, rows, K, K // 2 if ldc is None else ldc, K // 32, block, elem)


def _cfg(act=1, alpha=1.0):
    return mx.EpilogueCfgC(act, alpha)


A, W = _tensor(64, 96), _tensor(48, 96)
TAIL = ["r", "r_dtype", "ldr", "y", "y_dtype", "ldy", "stream"]
TAIL_OK = [P(16), 1, 48, P(16), 1, 48, None]
DENSE = (["a", "b", "cfg", "bias", "bias_dtype"] + TAIL, [A, W, _cfg(), P(16), 0] + TAIL_OK)
GROUPED = (["a", "off", "E", "b", "sc", "ss", "cfg", "bias", "bias_dtype", "bias_stride"] + TAIL,
           [A, P(16), 2, W, 2304, 144, _cfg(), P(16), 0, 48] + TAIL_OK)
CALLS = {"mx_linear": DENSE, "mx_linear_backward": DENSE, "mx_grouped_linear": GROUPED, "mx_grouped_linear_backward": GROUPED}


def call(lib, name, **kw):
    names, ok = CALLS[name]
    args = list(ok)
    for k, v in kw.items():
        args[names.index(k)] = v
    return getattr(lib, name)(*[B(a) if isinstance(a, ctypes.Structure) else a for a in args]), lib.mx_last_error()


@pytest.mark.parametrize("name", list(CALLS))
def test_refusals(lib, name):
    both = [dict(a=None), dict(b=None), dict(a=_tensor(64, 95)), dict(a=_tensor(64, 128)), dict(b=_tensor(48, 96, codes=17)),
            dict(b=_tensor(48, 96, elem=7)), dict(a=_tensor(-1, 96)), dict(cfg=_cfg(4)), dict(cfg=_cfg(-1)),
            dict(cfg=_cfg(0, 0.0)), dict(cfg=_cfg(0, NAN)), dict(cfg=_cfg(0, INF)), dict(bias_dtype=2), dict(bias=P(18)),
            dict(r_dtype=2), dict(r=P(17)), dict(ldr=47), dict(y=None), dict(y=P(17)), dict(y_dtype=2), dict(ldy=47)]
    if "grouped" in name:
        both += [dict(off=None), dict(off=P(18)), dict(E=0), dict(sc=-16), dict(ss=-1), dict(sc=8), dict(bias_stride=-1)]
    if "backward" in name:
        both += [dict(r=None), dict(cfg=None), dict(cfg=_cfg(3))]
    for kw in both:
        st, msg = call(lib, name, **kw)
        assert st == BAD and msg.startswith(name.encode()), (kw, st, msg)
    st, msg = call(lib, name, a=_tensor(2**31, 96))
    assert st == UNSUP, msg
    if "grouped" in name:
        assert call(lib, name, a=_tensor(64, 96, block=1))[0] == UNSUP
    assert call(lib, name, a=_tensor(0, 96), y=None, r=None if "backward" not in name else P(16))[0] == OK
    assert call(lib, name, b=_tensor(0, 96), y=None)[0] == OK


# ------------------------------------------------------------------ the binding
def operand(rows, K=64, experts=None):
    return mx.empty_mx(rows, K, "1d", device="cpu", experts=experts)


def f32(*shape):
    return torch.zeros(*shape)


OFF = torch.zeros(3, dtype=torch.int32)


@pytest.mark.parametrize("f", [
    lambda: mx.linear(operand(32), operand(48)), lambda: mx.linear_backward(operand(32), operand(48), f32(32, 48)),
    lambda: mx.grouped_linear(operand(32), OFF, operand(48, experts=2)),
    lambda: mx.grouped_linear_backward(operand(32), OFF, operand(48, experts=2), f32(32, 48))])
def test_host_operands_are_refused(monkeypatch, f):
    monkeypatch.setattr(mx, "_lib", StubLibrary())
    with pytest.raises(ValueError, match="CUDA"):
        f()


def _on(q, index=0):
    return mx.MXTensor(on(q.codes, index), on(q.scales, index), q.rows, q.K, q.block, q.elem)


@pytest.mark.parametrize("which", ["bias", "residual", "out", "offsets"])
@pytest.mark.parametrize("index", [-1, 1])
def test_other_devices_are_refused(monkeypatch, which, index):
    monkeypatch.setattr(mx, "_lib", StubLibrary())
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    at = {k: index if k == which else 0 for k in ("bias", "residual", "out", "offsets")}
    kw = dict(bias=on(f32(2, 48), at["bias"]), residual=on(f32(32, 48), at["residual"]), out=on(f32(32, 48), at["out"]))
    off = on(OFF, at["offsets"])
    monkeypatch.setattr(mx, "_check_offsets", lambda o, E: None)         # (it wants a real CUDA tensor)
    with pytest.raises(ValueError, match="one device|must be CUDA"):
        mx.grouped_linear(_on(operand(32)), off, _on(operand(48, experts=2)), **kw)


@pytest.mark.parametrize("match,kw", [
    ("residual must have shape", dict(residual=f32(32, 47))), ("residual must be", dict(residual=f32(32, 48).double())),
    ("residual must be row-major", dict(residual=f32(48, 32).t())), ("out must have shape", dict(out=f32(31, 48)))])
def test_binding_refuses(monkeypatch, match, kw):
    monkeypatch.setattr(mx, "_stream", lambda t, *others: 0)
    with pytest.raises(ValueError, match=match):
        mx.linear(operand(32), operand(48), **kw)


def test_unknown_activation(monkeypatch):
    monkeypatch.setattr(mx, "_stream", lambda t, *others: 0)
    with pytest.raises(KeyError):
        mx.linear(operand(32), operand(48), act="relu", out=f32(32, 48))
