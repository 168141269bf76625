"""Refusals of the feed-forward entry points: every call here is turned down
(or is a no-op) on the host, before anything is launched."""
import ctypes
import os

import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx

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


def _caller(lib, f, names, ok):
    def call(**kw):
        args = list(ok)
        for k, v in kw.items():
            args[names.index(k)] = v
        st = f(*args)
        return st, lib.mx_last_error()
    return call


def _gate(act=0, layout=0, alpha=1.0, limit=0.0, shift=0.0):
    return mx.GateCfgC(act, layout, alpha, limit, shift)


A, W = _tensor(64, 96), _tensor(96, 96)
GATE_ARGS = {
    "mx_gemm_gated": (["a", "b", "cfg", "h", "h_dtype", "ldh", "stream"], [A, W, _gate(), P(16), 1, 48, None]),
    "mx_gemm_gated_backward": (["a", "b", "cfg", "dh", "dh_dtype", "lddh", "h", "h_dtype", "ldh", "stream"],
                               [A, W, _gate(), P(16), 1, 48, P(16), 1, 96, None]),
    "mx_grouped_gemm_gated": (["a", "off", "E", "b", "sc", "ss", "cfg", "h", "h_dtype", "ldh", "stream"],
                              [A, P(16), 2, W, 4608, 288, _gate(), P(16), 1, 48, None]),
    "mx_grouped_gemm_gated_backward": (["a", "off", "E", "b", "sc", "ss", "cfg", "dh", "dh_dtype", "lddh", "h",
                                        "h_dtype", "ldh", "stream"],
                                       [A, P(16), 2, W, 4608, 288, _gate(), P(16), 1, 48, P(16), 1, 96, None]),
}


@pytest.mark.parametrize("name", list(GATE_ARGS))
def test_gated_rejects_bad_arguments(lib, name):
    names, ok = GATE_ARGS[name]
    ref = [B(v) if isinstance(v, ctypes.Structure) else v for v in ok]
    call = _caller(lib, getattr(lib, name), names, ref)
    st, msg = call(a=None)
    assert st == BAD and b"null" in msg
    st, msg = call(b=B(_tensor(96, 64)))
    assert st == BAD and b"A.K" in msg
    st, msg = call(b=B(_tensor(97, 96)))
    assert st == BAD and b"even" in msg
    st, msg = call(a=B(_tensor(64, 96, codes=8)))
    assert st == BAD and b"aligned" in msg
    st, msg = call(a=B(_tensor(64, 96, elem=9)))
    assert st == BAD and b"element type" in msg
    st, msg = call(cfg=None)
    assert st == BAD and b"null gate" in msg
    for act in (-1, 3):
        st, msg = call(cfg=B(_gate(act=act)))
        assert st == BAD and b"activation" in msg
    for layout in (-1, 2):
        st, msg = call(cfg=B(_gate(layout=layout)))
        assert st == BAD and b"layout" in msg
    for alpha in (0.0, -1.0, NAN, INF):
        st, msg = call(cfg=B(_gate(alpha=alpha)))
        assert st == BAD and b"alpha" in msg
    for limit in (-1.0, NAN):
        st, msg = call(cfg=B(_gate(limit=limit)))
        assert st == BAD and b"limit" in msg
    for shift in (NAN, INF):
        st, msg = call(cfg=B(_gate(shift=shift)))
        assert st == BAD and b"up_shift" in msg
    st, msg = call(h_dtype=2)
    assert st == BAD and b"dtype" in msg
    st, msg = call(h=None)
    assert st == BAD and b"null" in msg
    st, msg = call(h=P(17))
    assert st == BAD and b"aligned" in msg
    st, msg = call(ldh=47)
    assert st == BAD and b"stride" in msg
    st, msg = call(a=B(_tensor(1 << 31, 96)))
    assert st == UNSUP
    if "backward" in name:
        for kw in (dict(dh=None), dict(dh_dtype=7), dict(lddh=47), dict(dh=P(17)), dict(ldh=95)):
            assert call(**kw)[0] == BAD, kw
    if "grouped" in name:
        st, msg = call(a=B(_tensor(64, 96, block=1)))
        assert st == UNSUP and b"1-D" in msg
        for kw in (dict(off=None), dict(off=P(18)), dict(E=0), dict(sc=-16), dict(ss=-1), dict(sc=4600)):
            assert call(**kw)[0] == BAD, kw
    # empty: nothing to do, nothing dereferenced
    assert call(a=B(_tensor(0, 96)), h=None)[0] == OK
    assert call(b=B(_tensor(0, 96)), h=None)[0] == OK


def test_layer_norm_rejects_bad_arguments(lib):
    names = ["x", "dtype", "R", "C", "ldx", "w", "b", "w_dtype", "eps", "y", "ldy", "mean", "rstd", "stream"]
    call = _caller(lib, lib.mx_layer_norm, names,
                   (P(16), 1, 4, 33, 40, P(16), P(16), 0, 1e-5, P(16), 40, P(16), P(16), None))
    for kw, word in ((dict(dtype=2), b"dtype"), (dict(w_dtype=5), b"weight dtype"), (dict(R=-1), b"negative"),
                     (dict(C=-1), b"negative"), (dict(eps=-1.0), b"eps"), (dict(eps=NAN), b"eps"),
                     (dict(eps=INF), b"eps"), (dict(x=None), b"null x"), (dict(y=None), b"null y"),
                     (dict(ldx=32), b"stride"), (dict(ldy=32), b"stride"), (dict(x=P(17)), b"aligned"),
                     (dict(y=P(17)), b"aligned"), (dict(w=P(18)), b"aligned"), (dict(b=P(18)), b"aligned"),
                     (dict(mean=P(18)), b"aligned"), (dict(rstd=P(18)), b"aligned")):
        st, msg = call(**kw)
        assert st == BAD and word in msg, kw
    assert call(R=0, x=None, y=None)[0] == OK and call(C=0, x=None, y=None)[0] == OK


def test_layer_norm_backward_rejects_bad_arguments(lib):
    need = lib.mx_layer_norm_backward_workspace_size(4, 33)
    assert need >= 2 * 33 * 4
    assert lib.mx_layer_norm_backward_workspace_size(0, 33) == 0
    assert lib.mx_layer_norm_backward_workspace_size(4, 0) == 0
    names = ["dy", "x", "dtype", "R", "C", "lddy", "ldx", "mean", "rstd", "w", "w_dtype", "dx", "lddx", "dw", "db",
             "ws", "n", "stream"]
    call = _caller(lib, lib.mx_layer_norm_backward, names,
                   (P(16), P(16), 1, 4, 33, 40, 40, P(16), P(16), P(16), 0, P(16), 40, P(16), P(16), P(32), need,
                    None))
    for kw, word in ((dict(dtype=2), b"dtype"), (dict(w_dtype=5), b"weight dtype"), (dict(R=-1), b"negative"),
                     (dict(dy=None), b"null dy"), (dict(x=None), b"null x"), (dict(lddy=32), b"stride"),
                     (dict(ldx=32), b"stride"), (dict(lddx=32), b"stride"), (dict(dx=P(17)), b"aligned"),
                     (dict(mean=None), b"mean"), (dict(rstd=P(18)), b"rstd"), (dict(dw=P(18)), b"aligned"),
                     (dict(ws=None), b"workspace"), (dict(n=need - 1), b"workspace"), (dict(ws=P(24)), b"workspace")):
        st, msg = call(**kw)
        assert st == BAD and word in msg, kw
    assert call(C=0)[0] == OK


def test_dropout_rejects_bad_arguments(lib):
    names = ["x", "dtype", "R", "C", "ldx", "p", "seed", "offset", "r", "ldr", "y", "ldy", "stream"]
    call = _caller(lib, lib.mx_dropout, names, (P(16), 1, 4, 33, 40, 0.1, 1, 2, P(16), 40, P(16), 40, None))
    for kw, word in ((dict(dtype=2), b"dtype"), (dict(R=-1), b"negative"), (dict(p=-0.1), b"p must"),
                     (dict(p=1.1), b"p must"), (dict(p=NAN), b"p must"), (dict(x=None), b"null x"),
                     (dict(y=None), b"null y"), (dict(ldx=32), b"stride"), (dict(ldr=32), b"stride"),
                     (dict(ldy=32), b"stride"), (dict(x=P(17)), b"aligned"), (dict(r=P(17)), b"aligned")):
        st, msg = call(**kw)
        assert st == BAD and word in msg, kw
    assert call(R=0, x=None, y=None)[0] == OK


def test_binding_refuses_what_the_library_cannot_see(lib):
    """Host tensors, wrong shapes, types and strides raise before the call."""
    x = torch.zeros(4, 32)
    with pytest.raises(ValueError, match="CUDA"):
        mx.layer_norm(x)
    with pytest.raises(ValueError, match="CUDA"):
        mx.dropout(x, 0.1)
    with pytest.raises(ValueError, match="CUDA"):
        mx.layer_norm_backward(x, x, x[:, 0], x[:, 0])
    with pytest.raises(KeyError):
        mx.Gate(act="tanh").c_struct()
