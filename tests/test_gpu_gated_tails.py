"""The activations' relative accuracy, out in their tails too, where a bound on
the absolute error would say nothing.

The projections are exact here: a row of A holds two E4M3 values whose sum is
the gate projection (a float32 of 8 or 9 significant bits), every up
projection is 1.  What is left is the formula in float32 (U = 2^-24, hardware
exponential and reciprocal 2 U each):
  sigmoid(z)   5 U, and z's roundings: 2 U |z| for alpha x, 4 U |z| for the
               tanh form's cubic; one more U for what is rounded around it.
  GELU         q = Phi(-|x|): the fit and its evaluation 7 U, exponential and
               reciprocal 4 U, x^2 / 2's three roundings 1.25 U x^2; Phi itself
               adds one rounding where it is 1 - q.
The products around them add a U each; below 1e-37 the hardware flushes."""
import numpy as np
import pytest
import torch
from scipy.special import log_ndtr

import mxfp4_microscaling_quantization_mx_amd as mx
from oracle.gemm import dequant_f64
from gpu_util import banner, host, need_gpu, to_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def exact_gates(M, K=32):
    """An E4M3 operand [M, K] whose rows sum to exactly known gate projections,
    and those: both signs, 2^-12 to 2^5, more of them between 1/4 and 16."""
    rng = np.random.default_rng(M)
    mag = np.concatenate([2.0 ** rng.uniform(-12, 5, M // 2), 2.0 ** rng.uniform(-2, 4, M - M // 2)])
    e = np.floor(np.log2(mag)).astype(int)
    scale = (e - 4 + 127).astype(np.uint8)                  # values of 2^4 to 2^5 at scale 2^(e - 4)
    hi = rng.integers(8, 16, M)                             # 1.mmm: code (4 + 7) << 3 | mmm
    lo = rng.integers(8, 16, M)                             # 1.mmm * 2^-4 of it
    sign = rng.random(M) < 0.5
    sign[::2] = True                                        # most of them negative: the tails are there
    codes = np.zeros((M, K), np.uint8)
    codes[:, 0] = (sign * 128) | (11 << 3) | (hi - 8)
    codes[:, 1] = (sign * 128) | (7 << 3) | (lo - 8)
    x = np.where(sign, -1, 1) * (hi / 8 * 16 + lo / 8) * 2.0 ** (e - 4.0)
    assert np.array_equal(dequant_f64(codes, scale[:, None], "e4m3", "1d").sum(1), x)
    return mx.MXTensor(to_dev(codes), to_dev(np.repeat(scale[:, None], 4, 1))[:, :1], M, K, "1d", "e4m3"), x


def weights(N, K=32):
    """Gate and up rows of E4M3 1, 1, 0, ...: both projections of a row of A are
    the sum of its two values."""
    codes = np.zeros((2 * N, K), np.uint8)
    codes[:, :2] = 7 << 3
    return mx.MXTensor(to_dev(codes), to_dev(np.full((2 * N, 4), 127, np.uint8))[:, :1], 2 * N, K, "1d", "e4m3")


def reference(x, gate):
    """act(x), act'(x) and their tolerances."""
    if gate.act == "gelu":
        q = np.exp(log_ndtr(-np.abs(x)))
        cdf = np.where(x > 0, 1 - q, q)
        pdf = np.exp(-0.5 * x * x) / np.sqrt(2 * np.pi)
        tc = q * (11 + 1.25 * x * x) * U + np.where(x > 0, cdf * U, 0)
        a, d = x * cdf, cdf + x * pdf
        return a, np.abs(x) * tc + np.abs(a) * U, d, tc + np.abs(x * pdf) * (5 + 1.25 * x * x) * U + np.abs(d) * U
    if gate.act == "silu":
        z, dz, per = gate.alpha * x, gate.alpha, 2
    else:
        c = 2 * np.sqrt(2 / np.pi)
        z, dz, per = c * (x + 0.044715 * x ** 3), c * (1 + 3 * 0.044715 * x * x), 4
    s = 0.5 * (1 + np.tanh(z / 2))
    s = np.where(z < 0, np.exp(np.minimum(z, 0) - np.log1p(np.exp(np.minimum(z, 0)))), s)
    ts = s * (6 + per * np.abs(z)) * U
    a, one = x * s, 1 / (1 + np.exp(np.minimum(z, 700)))                     # 1 - s
    d = s + a * one * dz
    # 1 - s is a float32 subtraction from 1: off by s's error and one rounding
    td = ts + np.abs(x * dz) * (ts * one + s * (ts + U)) + np.abs(a * one * dz) * 6 * U + np.abs(d) * U
    return a, np.abs(x) * ts + np.abs(a) * U, d, td


@pytest.mark.parametrize("gate", [mx.Gate("gelu", up_shift=0.0), mx.Gate("gelu_tanh"), mx.Gate(),
                                  mx.Gate("silu", alpha=1.702)])
@pytest.mark.parametrize("M,N", [(600, 16), (420, 900), (1100, 3700)])
def test_relative_accuracy(gate, M, N):
    """On the kernel for few rows, the 128 x 64 tiles and the 256-row pipeline.
    The up projection equals the gate's, so h = act(g) g and, for dH = 1,
    dg = act'(g) g and du = act(g)."""
    need_gpu()
    qa, x = exact_gates(M)
    qb = weights(N)
    banner(f"gated tails {gate} {M}x{N}")
    h = host(mx.gemm_gated(qa, qb, gate, torch.float32)).astype(np.float64)
    dP = host(mx.gemm_gated_backward(qa, qb, torch.ones(M, N, device="cuda"), gate, torch.float32)).astype(np.float64)
    a, ta, d, td = reference(x, gate)
    for what, got, ref, tol in (("h", h, a * x, ta * np.abs(x)), ("dg", dP[:, 0::2], d * x, td * np.abs(x)),
                                ("du", dP[:, 1::2], a, ta)):
        assert np.array_equal(got, np.repeat(got[:, :1], N, 1)), what
        off = np.abs(got[:, 0] - ref) - (tol + np.abs(ref) * U + 1e-37)
        i = int(np.argmax(off))
        assert off[i] <= 0, f"{what} at {x[i]}: {got[i, 0]:.9e}, not {ref[i]:.9e} +- {tol[i]:.1e}"
