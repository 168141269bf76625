"""Layer norm where the mean is far above the spread: rows of one value, means
of 10^3 to 10^7 times the spread, and rows whose sum passes float32's range.

The mean is a double until it is subtracted, as a float32 and what that leaves,
so a centred value x' errs by its own two roundings and 3 2^-48 |mean|, and what
follows is what float32 makes of exact centred values: with depth the longest
chain of additions of a row, the variance errs by (depth + 6) 2^-24 of itself
and by the centred values' errors.  Rows of one value have exact sums (24 bits
times C below 2^29), so nothing is left of them."""
import numpy as np
import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx
from gpu_util import banner, host, need_gpu
from test_gpu_norm import BF, F32, U, backward, f64, near, strided

pytestmark = pytest.mark.gpu

# widths of one wave, 16-byte pieces, single elements, many waves, past the registers
WIDTHS = [1, 8, 64, 100, 1111, 2880, 9000, 12289, 16384, 70001]


def exact(x, w, b, eps):
    """y, mean, rstd in float64 and their tolerances."""
    C = x.shape[1]
    depth = C / 64 + 16
    mean = x.mean(1, keepdims=True)
    xc = x - mean
    xc = xc - xc.mean(1, keepdims=True)
    var = (xc * xc).mean(1, keepdims=True)
    rstd = (var + eps) ** -0.5
    left = 3 * 2.0 ** -48 * np.abs(mean)
    ec = 2 * U * np.abs(xc) + left
    ev = (depth + 6) * U * var + 2 * left * np.abs(xc).mean(1, keepdims=True) + left ** 2
    rel = 0.5 * ev / (var + eps) + 4 * U
    xh = xc * rstd
    ty = np.abs(w) * rstd * ec + np.abs(w * xh) * (rel + 8 * U) + 8 * U * np.abs(b)
    return (xh * w + b, mean[:, 0], rstd[:, 0]), (2 * ty, (U + 2.0 ** -48) * np.abs(mean[:, 0]), (2 * rel * rstd)[:, 0])


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("pad,lead", [(0, 0), (3, 1)])
def test_rows_of_one_value(C, dtype, pad, lead):
    """y is the bias and rstd 1 / sqrt(eps) whatever the value."""
    need_gpu()
    vals = np.array([12345.678, -1e6, 0.1, -3.3e-5, 7.7e9, 1e37, -3e38, 0.0])
    x = strided(np.repeat(vals[:, None], C, 1), dtype, pad, lead)
    b = torch.linspace(-1, 1, C, device="cuda")
    banner(f"norm of one value C={C} {dtype} pad {pad}")
    y, mean, rstd = mx.layer_norm(x, None, b, 1e-5, out=strided(np.zeros((len(vals), C)), dtype, pad, lead))
    assert torch.equal(y, b.to(dtype).expand_as(y))
    assert torch.equal(mean, x[:, 0].float())
    assert np.abs(host(rstd) * np.sqrt(np.float64(np.float32(1e-5))) - 1).max() < 4 * U


@pytest.mark.parametrize("C", WIDTHS[2:])
@pytest.mark.parametrize("pad,lead", [(0, 0), (3, 1)])
def test_mean_far_above_the_spread(C, pad, lead):
    need_gpu()
    rng = np.random.default_rng(C)
    means = np.array([0.0, 1e3, -1e4, 1e5, -1e6, 1e7, 3e4, 2e37])
    spread = np.array([1.0, 1.0, 1.0, 1.0, 1.0, 10.0, 1e-2, 1e32])
    x = means[:, None] + spread[:, None] * rng.standard_normal((len(means), C))
    xd = strided(x, F32, pad, lead)
    w, b = 1 + 0.1 * rng.standard_normal(C), 0.1 * rng.standard_normal(C)
    wd, bd = (torch.from_numpy(t.astype(np.float32)).cuda() for t in (w, b))
    xs = f64(xd)
    xs[-1] = 0.0                                  # its variance is past float32: only its mean is held to
    banner(f"norm far mean C={C} pad {pad}")
    y, mean, rstd = mx.layer_norm(xd, wd, bd)
    (ry, rm, rr), (ty, tm, tr) = exact(xs, f64(wd), f64(bd), 1e-5)
    big = f64(xd)[-1].mean()
    near(host(y)[:-1], ry[:-1], ty[:-1], "y")
    near(host(mean)[:-1], rm[:-1], tm[:-1], "mean")
    near(host(rstd)[:-1], rr[:-1], tr[:-1], "rstd")
    assert abs(host(mean)[-1].astype(np.float64) - big) <= (U + 2.0 ** -48) * abs(big)


def test_bf16_means_far_above_the_spread():
    """bf16 rows of two neighbouring values."""
    need_gpu()
    rng = np.random.default_rng(5)
    x = np.where(rng.random((6, 2880)) < 0.3, 2.0 ** np.arange(6)[:, None] * 128, 2.0 ** np.arange(6)[:, None] * 129)
    xd = strided(x, BF, 0, 0)
    banner("norm bf16 far mean")
    y, mean, rstd = mx.layer_norm(xd)
    (ry, rm, rr), (ty, tm, tr) = exact(f64(xd), np.ones(2880), np.zeros(2880), 1e-5)
    near(host(y.float()), ry, ty, "y", True)
    near(host(mean), rm, tm, "mean")
    near(host(rstd), rr, tr, "rstd")


@pytest.mark.parametrize("C", [5, 64, 100, 1111, 2880, 9000])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_backward_of_huge_rows_of_one_value(C, dtype):
    """mean * rstd is past float32, the centred values are zero: the lanes past
    the row's end must not bring an infinity into its sums."""
    need_gpu()
    rng = np.random.default_rng(C)
    vals = np.array([2.0 ** 123, -3e38, 1e30, -1e36])
    x = strided(np.repeat(vals[:, None], C, 1), dtype, 0, 0)
    dy = strided(rng.standard_normal((len(vals), C)), dtype, 0, 0)
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal(C)).astype(np.float32)).cuda()
    banner(f"norm backward of huge rows C={C} {dtype}")
    _, mean, rstd = mx.layer_norm(x, w)
    got = mx.layer_norm_backward(dy, x, mean, rstd, w)
    ref, tol = backward(f64(dy), f64(x), f64(mean), f64(rstd), f64(w))
    near(host(got[0].float()), ref[0], tol[0], "dx", dtype == BF)
    near(host(got[1]), ref[1], tol[1], "dweight")
    near(host(got[2]), ref[2], tol[2], "dbias")


def test_rows_without_columns():
    """The mean of nothing is NaN, not what the memory held."""
    need_gpu()
    banner("norm no columns")
    stale = [torch.full((5,), 3.0, device="cuda") for _ in range(2)]
    del stale
    y, mean, rstd = mx.layer_norm(torch.empty(5, 0, device="cuda"))
    assert y.shape == (5, 0) and mean.isnan().all() and rstd.isnan().all()
    dx, dw, db = mx.layer_norm_backward(y, y, mean, rstd)
    assert dx.shape == (5, 0) and dw.shape == db.shape == (0,)
