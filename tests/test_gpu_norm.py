"""Layer norm and its backward pass against the formulas in float64.

Tolerances: a float32 sum of n terms in parallel parts errs by at most depth *
2^-24 * sum|terms|, depth the longest chain of additions: at most C / 64 + 16
along a row and min(R, R / 64 + 128) over the rows.  The other steps add a few
roundings of 2^-24 each; bf16 outputs half an ulp.
"""
import numpy as np
import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx
from gpu_util import banner, bf16_half_ulp, host, need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def strided(a, dtype, pad, lead):
    """A device copy of a [R, C] with row stride C + pad, `lead` elements into
    its buffer."""
    R, C = a.shape
    buf = torch.full((R * (C + pad) + lead + 1,), 9.0, dtype=dtype, device="cuda")
    t = buf[lead:lead + R * (C + pad)].view(R, C + pad)[:, :C]
    t.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(dtype))
    return t


def f64(t):
    return t.double().cpu().numpy()


def near(got, ref, tol, what, bf16=False):
    got = np.asarray(got, dtype=np.float64)
    if bf16:
        tol = tol + bf16_half_ulp(np.abs(ref) + tol)
    over = np.abs(got - ref) - tol
    assert np.all(over <= 0), f"{what}: {int((over > 0).sum())} of {over.size} off, worst by {over.max():.3e}"


def forward(x, w, b, eps):
    """y, mean, rstd in float64 and their tolerances."""
    C = x.shape[1]
    depth = C / 64 + 16
    mean = x.mean(1)
    xc = x - mean[:, None]
    var = (xc * xc).mean(1)
    rstd = (var + eps) ** -0.5
    em = depth * U * np.abs(x).mean(1)
    rel = 0.5 * (em ** 2 + (depth + 4) * U * var) / (var + eps) + 4 * U
    xh = xc * rstd[:, None]
    ty = np.abs(w) * (rstd * em)[:, None] + np.abs(w * xh) * (rel[:, None] + 8 * U) + 8 * U * np.abs(b)
    return (xh * w + b, mean, rstd), (2 * ty, 2 * em + U * np.abs(mean), 2 * rel * rstd)


def backward(dy, x, mean, rstd, w):
    R, C = x.shape
    depth, rows = C / 64 + 16, min(R, R / 64 + 128)
    rs = rstd[:, None]
    xh = (x - mean[:, None]) * rs
    gy = dy * w
    s1, s2 = gy.mean(1, keepdims=True), (gy * xh).mean(1, keepdims=True)
    e1 = (depth + 2) * U * np.abs(gy).mean(1, keepdims=True)
    e2 = (depth + 5) * U * np.abs(gy * xh).mean(1, keepdims=True)
    dx = rs * (gy - s1 - xh * s2)
    tx = rs * (e1 + np.abs(xh) * e2 + 8 * U * (np.abs(gy) + np.abs(s1) + np.abs(xh * s2)))
    tw, tb = (rows + 6) * U * np.abs(dy * xh).sum(0), (rows + 2) * U * np.abs(dy).sum(0)
    return (dx, (dy * xh).sum(0), dy.sum(0)), (2 * tx, tw, tb)


SHAPES = [(1, 1), (1, 2880), (3, 7), (5, 64), (64, 2880), (33, 1111), (1000, 100), (517, 41), (2, 5000), (7, 4096),
          (3, 12289), (9, 16384), (2, 24584), (2, 70001), (2500, 256), (4100, 72)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("dtype,wtype", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("pad,lead", [(0, 0), (8, 8), (3, 1)])
def test_forward_and_backward(R, C, dtype, wtype, pad, lead):
    """One row and one column to long rows and many rows; rows contiguous,
    padded and starting at odd elements."""
    need_gpu()
    rng = np.random.default_rng([R, C, pad])
    x = rng.standard_normal((R, C)) * rng.uniform(0.5, 2.5, (R, 1)) + rng.standard_normal((R, 1))
    xd = strided(x, dtype, pad, lead)
    w = torch.from_numpy(1 + 0.1 * rng.standard_normal(C)).to(wtype).cuda()
    b = torch.from_numpy(0.1 * rng.standard_normal(C)).to(wtype).cuda()
    banner(f"norm {R}x{C} {dtype} {wtype} pad {pad}")
    out = strided(np.zeros((R, C)), dtype, pad, lead)
    y, mean, rstd = mx.layer_norm(xd, w, b, eps=1e-5, out=out)
    (ry, rm, rr), (ty, tm, tr) = forward(f64(xd), f64(w), f64(b), 1e-5)
    near(host(y.float()), ry, ty, "y", dtype == BF)
    near(host(mean), rm, tm, "mean")
    near(host(rstd), rr, tr, "rstd")
    assert torch.all(out._base[:lead] == 9.0) and out._base[-1] == 9.0

    dy = strided(rng.standard_normal((R, C)) * 0.1, dtype, pad, lead)
    dx = strided(np.zeros((R, C)), dtype, pad, lead)
    got = mx.layer_norm_backward(dy, xd, mean, rstd, w, out=dx)
    ref, tol = backward(f64(dy), f64(xd), f64(mean), f64(rstd), f64(w))
    near(host(got[0].float()), ref[0], tol[0], "dx", dtype == BF)
    near(host(got[1].float()), ref[1], tol[1], "dweight", wtype == BF)
    near(host(got[2].float()), ref[2], tol[2], "dbias", wtype == BF)
    assert torch.all(dx._base[:lead] == 9.0) and dx._base[-1] == 9.0
    if pad:
        assert torch.all(dx._base[lead:lead + R * (C + pad)].view(R, C + pad)[:, C:] == 9.0)


@pytest.mark.parametrize("R,C", [(64, 2880), (33, 1111), (5, 9000)])
def test_without_weight_and_in_place(R, C):
    """No weight and no bias; bias alone; y over x, dx over dy and over x."""
    need_gpu()
    rng = np.random.default_rng(R)
    x = rng.standard_normal((R, C)) + 2
    banner(f"norm in place {R}x{C}")
    xd = strided(x, F32, 0, 0)
    one, zero = np.ones(C), np.zeros(C)
    y, mean, rstd = mx.layer_norm(xd, eps=0.0)
    (ry, _, _), (ty, _, _) = forward(f64(xd), one, zero, 0.0)
    near(host(y), ry, ty, "y")
    b = torch.from_numpy(rng.standard_normal(C)).to(BF).cuda()
    (ry, _, _), (ty, _, _) = forward(f64(xd), one, f64(b), 1e-5)
    z = xd.clone()
    assert mx.layer_norm(z, None, b, out=z)[0] is z
    near(host(z), ry, ty, "y over x")
    dy = strided(rng.standard_normal((R, C)), F32, 0, 0)
    ref, tol = backward(f64(dy), f64(xd), f64(mean), f64(rstd), one)
    for over in (dy.clone(), xd.clone()):
        d, xx = (over, xd) if over.data_ptr() and torch.equal(over, dy) else (dy, over)
        got = mx.layer_norm_backward(d, xx, mean, rstd, out=over)
        near(host(over), ref[0], tol[0], "dx in place")
        near(host(got[1]), ref[1], tol[1], "dweight")
        near(host(got[2]), ref[2], tol[2], "dbias")


@pytest.mark.parametrize("C", [2880, 1111, 9000])
def test_far_mean_and_constant_rows(C):
    """A mean 10^4 times the spread (a difference of sums would lose it) and
    rows of one value, whose variance is zero."""
    need_gpu()
    rng = np.random.default_rng(2)
    x = rng.standard_normal((6, C)) + 1e4
    x[2], x[3], x[4] = 0.0, 3.25, -1e6
    xd = strided(x, F32, 0, 0)
    banner(f"norm far mean {C}")
    y, mean, rstd = mx.layer_norm(xd)
    (ry, rm, rr), (ty, tm, tr) = forward(f64(xd), np.ones(C), np.zeros(C), 1e-5)
    near(host(y), ry, ty, "y")
    near(host(mean), rm, tm, "mean")
    near(host(rstd), rr, tr, "rstd")


@pytest.mark.parametrize("R,C", [(40, 2880), (40, 1111), (12, 9000)])
def test_nan_and_inf_stay_in_their_rows(R, C):
    need_gpu()
    rng = np.random.default_rng(4)
    x = rng.standard_normal((R, C))
    x[3, 5], x[7, C - 1], x[11, 0] = np.nan, np.inf, -np.inf
    banner(f"norm nan {R}x{C}")
    y, mean, rstd = mx.layer_norm(strided(x, BF, 0, 0))
    bad = np.zeros(R, bool)
    bad[[3, 7, 11]] = True
    y = host(y.float())
    assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()
    dy = rng.standard_normal((R, C))
    dx, dw, db = mx.layer_norm_backward(strided(dy, BF, 0, 0), strided(x, BF, 0, 0), mean, rstd)
    dx = host(dx.float())
    assert np.isnan(dx[bad]).all() and np.isfinite(dx[~bad]).all()
    assert np.isnan(host(dw)).all() and np.isfinite(host(db)).all()


def test_no_rows():
    need_gpu()
    banner("norm no rows")
    x = torch.empty(0, 72, device="cuda")
    y, mean, rstd = mx.layer_norm(x)
    assert y.shape == (0, 72)
    _, dw, db = mx.layer_norm_backward(x, x, mean, rstd)
    assert torch.all(dw == 0) and torch.all(db == 0)


@pytest.mark.parametrize("C", [72, 101])
def test_backward_against_differences(C):
    """dx, dweight and dbias against central differences of sum(y dy) in
    float64."""
    need_gpu()
    rng = np.random.default_rng(6)
    R = 3
    x, w, b = rng.standard_normal((R, C)), 1 + 0.2 * rng.standard_normal(C), 0.1 * rng.standard_normal(C)
    dy = rng.standard_normal((R, C))
    cast = lambda a: a.astype(np.float32).astype(np.float64)
    x, w, b, dy = cast(x), cast(w), cast(b), cast(dy)
    dev = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()
    banner(f"norm differences {C}")
    _, mean, rstd = mx.layer_norm(dev(x), dev(w), dev(b))
    dx, dw, db = (host(t) for t in mx.layer_norm_backward(dev(dy), dev(x), mean, rstd, dev(w)))
    loss = lambda x, w, b: float((forward(x, w, b, 1e-5)[0][0] * dy).sum())
    h = 1e-5

    def diff(i, at):
        hi, lo = [x.copy(), w.copy(), b.copy()], [x.copy(), w.copy(), b.copy()]
        hi[i][at] += h
        lo[i][at] -= h
        return (loss(*hi) - loss(*lo)) / (2 * h)

    for c in range(0, C, 7):
        assert abs(diff(0, (1, c)) - dx[1, c]) < 2e-5
        assert abs(diff(1, c) - dw[c]) < 2e-5 and abs(diff(2, c) - db[c]) < 2e-5


@pytest.mark.parametrize("R,C,dtype", [(4099, 1111, F32), (16384, 2880, BF), (300, 9000, BF)])
def test_same_bits_every_run(R, C, dtype):
    """Sums in a fixed order: equal bits from run to run and on another
    stream."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(R, C, device="cuda", generator=g).to(dtype)
    dy = torch.randn(R, C, device="cuda", generator=g).to(dtype)
    banner(f"norm repeat {R}x{C}")
    one = mx.layer_norm(x) + mx.layer_norm_backward(dy, x, *mx.layer_norm(x)[1:])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        two = mx.layer_norm(x) + mx.layer_norm_backward(dy, x, *mx.layer_norm(x)[1:])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(one, two))
    ref, tol = backward(f64(dy), f64(x), f64(one[1]), f64(one[2]), np.ones(C))
    near(host(one[4]), ref[1], tol[1], "dweight")
    near(host(one[5]), ref[2], tol[2], "dbias")


def test_graph_replays_equal_eager_calls():
    """A captured forward and backward pass, replayed between eager calls."""
    need_gpu()
    x, dy = torch.randn(1000, 2880, device="cuda"), torch.randn(1000, 2880, device="cuda")
    w, b = torch.randn(2880, device="cuda"), torch.randn(2880, device="cuda")

    def run():
        f = mx.layer_norm(x, w, b)
        return f + mx.layer_norm_backward(dy, x, f[1], f[2], w) + (mx.dropout(x, 0.3, 5, 6, residual=dy),)

    banner("norm and dropout graph")
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for k in range(3):
        x.normal_()
        dy.normal_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, run())), k
