"""Refusals of the expert layer's entry points: every call here is turned down
(or is a no-op) on the host, before anything is launched."""
import ctypes
import os

import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx

P, B = ctypes.c_void_p, ctypes.byref
BAD, UNSUP, OK = mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED, mx.MX_OK
NAN, INF = float("nan"), float("inf")
BIG = 2**31


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mx.LIB_PATH):
        pytest.skip("libmxfp4.so not built")
    return mx.load_library()


def _router(score=0, renorm=1, scale=1.0):
    return mx.RouterCfgC(score, renorm, scale)


# entry point -> argument names and a valid call
CALLS = {
    "mx_route": (["x", "dtype", "T", "E", "ld", "top", "cfg", "ids", "w", "stream"],
                 [P(16), 1, 4, 32, 32, 4, _router(), P(16), P(16), None]),
    "mx_route_backward": (["dw", "x", "dtype", "T", "E", "ld", "ids", "top", "cfg", "dx", "ldd", "stream"],
                          [P(16), P(16), 1, 4, 32, 32, P(16), 4, _router(), P(16), 32, None]),
    "mx_expert_sort": (["ids", "T", "top", "E", "offsets", "rows", "dest", "ws", "nws", "stream"],
                       [P(16), 2048, 4, 32, P(16), P(16), P(16), P(16), 3 * 32 * 4, None]),
    "mx_expert_dispatch": (["x", "dtype", "T", "C", "ldx", "dest", "top", "xs", "rows", "ldxs", "stream"],
                           [P(16), 1, 4, 64, 64, P(16), 2, P(16), 8, 64, None]),
    "mx_expert_combine": (["y", "dtype", "rows", "C", "ldy", "dest", "w", "T", "top", "r", "ldr", "out", "ldo", "stream"],
                          [P(16), 1, 8, 64, 64, P(16), P(16), 4, 2, P(16), 64, P(16), 64, None]),
    "mx_expert_combine_backward": (["dout", "dtype", "T", "C", "lddo", "y", "rows", "ldy", "dest", "w", "top", "dy",
                                    "lddy", "dw", "stream"],
                                   [P(16), 1, 4, 64, 64, P(16), 8, 64, P(16), P(16), 2, P(16), 64, P(16), None]),
    "mx_bias_grad": (["dp", "dtype", "M", "N", "ld", "out", "odtype", "ws", "nws", "stream"],
                     [P(16), 1, 2000, 64, 64, P(16), 0, P(16), 1 << 20, None]),
    "mx_grouped_bias_grad": (["dp", "dtype", "M", "N", "ld", "off", "E", "out", "odtype", "ws", "nws", "stream"],
                             [P(16), 1, 2000, 64, 64, P(16), 3, P(16), 0, P(16), 1 << 20, None]),
}


def call(lib, name, **kw):
    names, ok = CALLS[name]
    args = list(ok)
    for k, v in kw.items():
        args[names.index(k)] = v
    return getattr(lib, name)(*[B(a) if isinstance(a, ctypes.Structure) else a for a in args]), lib.mx_last_error()


REFUSED = [
    ("mx_route", BAD, dict(dtype=2)), ("mx_route", BAD, dict(T=-1)), ("mx_route", BAD, dict(E=0)),
    ("mx_route", BAD, dict(top=0)), ("mx_route", BAD, dict(top=33)), ("mx_route", BAD, dict(ld=31)),
    ("mx_route", BAD, dict(x=None)), ("mx_route", BAD, dict(x=P(17))), ("mx_route", BAD, dict(ids=None)),
    ("mx_route", BAD, dict(ids=P(18))), ("mx_route", BAD, dict(w=None)), ("mx_route", BAD, dict(w=P(18))),
    ("mx_route", BAD, dict(cfg=None)), ("mx_route", BAD, dict(cfg=_router(2))), ("mx_route", BAD, dict(cfg=_router(0, 2))),
    ("mx_route", BAD, dict(cfg=_router(scale=NAN))), ("mx_route", BAD, dict(cfg=_router(scale=INF))),
    ("mx_route", UNSUP, dict(E=1025, ld=1025)), ("mx_route", UNSUP, dict(E=128, ld=128, top=65)),
    ("mx_route", UNSUP, dict(T=BIG)), ("mx_route", UNSUP, dict(T=2**26 - 3)),
    ("mx_route_backward", UNSUP, dict(T=2**26 - 3)),
    ("mx_route_backward", BAD, dict(dw=None)), ("mx_route_backward", BAD, dict(dw=P(18))),
    ("mx_route_backward", BAD, dict(ids=None)), ("mx_route_backward", BAD, dict(dx=None)),
    ("mx_route_backward", BAD, dict(ldd=31)), ("mx_route_backward", BAD, dict(dx=P(17))),
    ("mx_route_backward", BAD, dict(top=33)), ("mx_route_backward", BAD, dict(x=None)),
    ("mx_route_backward", UNSUP, dict(E=2000, ld=2000, ldd=2000)),
    ("mx_expert_sort", BAD, dict(T=-1)), ("mx_expert_sort", BAD, dict(top=0)), ("mx_expert_sort", BAD, dict(E=0)),
    ("mx_expert_sort", BAD, dict(ids=None)), ("mx_expert_sort", BAD, dict(ids=P(18))),
    ("mx_expert_sort", BAD, dict(offsets=None)), ("mx_expert_sort", BAD, dict(rows=None)),
    ("mx_expert_sort", BAD, dict(dest=None)), ("mx_expert_sort", BAD, dict(dest=P(18))),
    ("mx_expert_sort", BAD, dict(ws=None)), ("mx_expert_sort", BAD, dict(ws=P(18))),
    ("mx_expert_sort", BAD, dict(nws=3 * 32 * 4 - 1)),
    ("mx_expert_sort", UNSUP, dict(E=1025)), ("mx_expert_sort", UNSUP, dict(T=BIG // 4)),
    ("mx_expert_dispatch", BAD, dict(dtype=5)), ("mx_expert_dispatch", BAD, dict(T=-1)),
    ("mx_expert_dispatch", BAD, dict(C=-1)), ("mx_expert_dispatch", BAD, dict(rows=-1)),
    ("mx_expert_dispatch", BAD, dict(top=0)), ("mx_expert_dispatch", BAD, dict(dest=None)),
    ("mx_expert_dispatch", BAD, dict(x=None)), ("mx_expert_dispatch", BAD, dict(xs=None)),
    ("mx_expert_dispatch", BAD, dict(ldx=63)), ("mx_expert_dispatch", BAD, dict(ldxs=63)),
    ("mx_expert_dispatch", BAD, dict(xs=P(17))), ("mx_expert_dispatch", UNSUP, dict(T=BIG)),
    ("mx_expert_dispatch", UNSUP, dict(T=1 << 30, C=1024, ldx=1024, ldxs=1024)),
    ("mx_expert_dispatch", UNSUP, dict(T=2**26 - 3)), ("mx_expert_combine", UNSUP, dict(T=2**26 - 3)),
    ("mx_expert_combine", UNSUP, dict(T=2**25, C=513, ldy=513, ldr=513, ldo=513)),
    ("mx_expert_combine_backward", UNSUP, dict(dtype=0, T=2**25, C=257, ldy=257, lddo=257, lddy=257)),
    ("mx_expert_combine", BAD, dict(dtype=2)), ("mx_expert_combine", BAD, dict(rows=-1)),
    ("mx_expert_combine", BAD, dict(top=0)), ("mx_expert_combine", BAD, dict(y=None)),
    ("mx_expert_combine", BAD, dict(y=P(17))), ("mx_expert_combine", BAD, dict(ldy=63)),
    ("mx_expert_combine", BAD, dict(dest=None)), ("mx_expert_combine", BAD, dict(dest=P(18))),
    ("mx_expert_combine", BAD, dict(w=P(18))), ("mx_expert_combine", BAD, dict(r=P(17))),
    ("mx_expert_combine", BAD, dict(ldr=63)), ("mx_expert_combine", BAD, dict(out=None)),
    ("mx_expert_combine", BAD, dict(ldo=63)),
    ("mx_expert_combine_backward", BAD, dict(dout=None)), ("mx_expert_combine_backward", BAD, dict(y=None)),
    ("mx_expert_combine_backward", BAD, dict(dy=None)), ("mx_expert_combine_backward", BAD, dict(w=None)),
    ("mx_expert_combine_backward", BAD, dict(dw=None)), ("mx_expert_combine_backward", BAD, dict(dw=P(18))),
    ("mx_expert_combine_backward", BAD, dict(lddo=63)), ("mx_expert_combine_backward", BAD, dict(lddy=63)),
    ("mx_expert_combine_backward", BAD, dict(ldy=63)), ("mx_expert_combine_backward", BAD, dict(dest=None)),
    ("mx_bias_grad", BAD, dict(dtype=2)), ("mx_bias_grad", BAD, dict(odtype=2)), ("mx_bias_grad", BAD, dict(M=-1)),
    ("mx_bias_grad", BAD, dict(N=-1)), ("mx_bias_grad", BAD, dict(dp=None)), ("mx_bias_grad", BAD, dict(dp=P(17))),
    ("mx_bias_grad", BAD, dict(ld=63)), ("mx_bias_grad", BAD, dict(out=None)), ("mx_bias_grad", BAD, dict(out=P(18))),
    ("mx_bias_grad", BAD, dict(ws=None)), ("mx_bias_grad", BAD, dict(ws=P(18))), ("mx_bias_grad", BAD, dict(nws=64)),
    ("mx_bias_grad", UNSUP, dict(M=BIG)), ("mx_bias_grad", UNSUP, dict(M=2**30)),
    ("mx_bias_grad", UNSUP, dict(M=0, N=2**30, ld=2**30)), ("mx_grouped_bias_grad", UNSUP, dict(M=2**30 - 512)),
    ("mx_grouped_bias_grad", BAD, dict(off=None)), ("mx_grouped_bias_grad", BAD, dict(off=P(18))),
    ("mx_grouped_bias_grad", BAD, dict(E=0)), ("mx_grouped_bias_grad", BAD, dict(nws=64)),
]


@pytest.mark.parametrize("name,status,change", REFUSED, ids=lambda v: str(v) if not isinstance(v, dict) else
                         ",".join(f"{k}" for k in v))
def test_refused(lib, name, status, change):
    st, msg = call(lib, name, **change)
    assert st == status, (st, msg)
    assert msg.startswith(name.encode())


@pytest.mark.parametrize("name,change", [
    ("mx_route", dict(T=0, x=None, ids=None, w=None)), ("mx_route_backward", dict(T=0, x=None, dx=None, ids=None, dw=None)),
    ("mx_expert_dispatch", dict(T=0, x=None, dest=None)), ("mx_expert_dispatch", dict(C=0, x=None, xs=None)),
    ("mx_expert_dispatch", dict(rows=0, xs=None)), ("mx_expert_combine", dict(T=0, out=None, dest=None)),
    ("mx_expert_combine", dict(C=0, out=None)), ("mx_expert_combine_backward", dict(T=0, dout=None, dw=None)),
    ("mx_bias_grad", dict(N=0, dp=None, out=None)), ("mx_grouped_bias_grad", dict(N=0, dp=None, out=None))])
def test_no_ops(lib, name, change):
    assert call(lib, name, **change) == (OK, b"")


def test_workspace_sizes(lib):
    f = lib.mx_expert_sort_workspace_size
    assert f(1024, 4, 32) == 0 and f(1025, 4, 32) == 3 * 32 * 4 and f(16384, 4, 32) == 17 * 32 * 4
    assert f(0, 4, 32) == f(-1, 4, 32) == f(4, 0, 32) == f(4, 4, 0) == f(4, 4, 1025) == f(BIG, 4, 32) == 0
    f = lib.mx_bias_grad_workspace_size
    assert f(1024, 2880, 32) == 0 and f(0, 8, 1) == f(8, 0, 1) == f(1100, 8, 0) == f(BIG, 8, 1) == 0
    for M, N, E in ((1025, 7, 1), (2048, 64, 1), (65536, 2880, 32)):
        tiles = M // 256 + min(E, M)                       # a partial tile per expert at most
        assert f(M, N, E) == tiles * N * 4


# ------------------------------------------------------------------ the binding's own checks (no library call)
def f32(*shape):
    return torch.zeros(*shape)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.mark.parametrize("match,f", [
    ("logits must be", lambda: mx.route(i32(2, 4), 1)),
    ("row-major", lambda: mx.route(f32(4, 3).t(), 1)),
    ("ids must be", lambda: mx.route_backward(f32(2, 1), f32(2, 4), f32(2, 1))),
    ("dweights must have shape", lambda: mx.route_backward(f32(2, 2), f32(2, 4), i32(2, 1))),
    ("ids must have 2 rows", lambda: mx.route_backward(f32(3, 1), f32(2, 4), i32(3, 1))),
    ("ids must be", lambda: mx.expert_sort(i32(4), 3)),
    ("ids must be", lambda: mx.expert_sort(i32(4, 4)[:, :2], 3)),
    ("ids must be", lambda: mx.expert_sort(torch.zeros(4, 2, dtype=torch.int64), 3)),
    ("dest must have 3 rows", lambda: mx.expert_dispatch(f32(3, 8), i32(4, 2))),
    ("dest must be", lambda: mx.expert_combine(f32(3, 8), i32(4))),
    ("weights must have shape", lambda: mx.expert_combine(f32(3, 8), i32(4, 2), f32(4, 1))),
    ("weights must be", lambda: mx.expert_combine(f32(3, 8), i32(4, 2), f32(4, 2).double())),
    ("residual must have shape", lambda: mx.expert_combine(f32(3, 8), i32(4, 2), residual=f32(4, 9))),
    ("residual must be", lambda: mx.expert_combine(f32(3, 8), i32(4, 2), residual=f32(4, 8).bfloat16())),
    ("dout must have shape", lambda: mx.expert_combine_backward(f32(3, 8), f32(3, 8), i32(4, 2), f32(4, 2))),
    ("dp must be", lambda: mx.bias_grad(f32(8))),
    ("dtype must be", lambda: mx.bias_grad(f32(8, 8), dtype=torch.float16)),
])
def test_binding_refuses(lib, match, f):
    with pytest.raises(ValueError, match=match):
        f()


def test_unknown_score():
    with pytest.raises(KeyError):
        mx.Router("relu").c_struct()
