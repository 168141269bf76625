"""The linear layer's backward pass against central differences of an activation
written here in float64 from its definition (the derivative appears nowhere)."""
import math

import numpy as np
import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx
from gpu_util import banner, host, need_gpu, to_dev
from test_gpu_linear_epilogue import grouped, operand, projections

pytestmark = pytest.mark.gpu
F32 = torch.float32
U = 2.0 ** -24
H = 1e-4
PHI = np.vectorize(lambda x: 0.5 * math.erfc(-x * math.sqrt(0.5)))


def value(x, act, alpha):
    if act == "silu":
        return x / (1 + np.exp(-alpha * x))
    if act == "gelu":
        return x * PHI(x)
    return 0.5 * x * (1 + np.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))


def check_slope(dp, dy, P, err, act, alpha):
    """dp against dy times the difference quotient at P.  The quotient errs by H^2 / 6 times
    a third derivative (below 4 for alpha up to 2) and by the float64 roundings of two
    values, a few 2^-53 (1 + |P|) each, over 2 H.  The kernel's point errs by err, times a
    second derivative (at most 0.85 max(1, alpha)), its derivative by 128 of 2^-24 (the
    exponential's error with |z| up to 35, where the slope is not yet constant) and the
    product with dy by one rounding of at most 1.13 |dy|."""
    quotient = (value(P + H, act, alpha) - value(P - H, act, alpha)) / (2 * H)
    tol = 4 * H * H / 6 + 1e-15 * (1 + np.abs(P)) / H + 0.85 * max(1.0, alpha) * err + (128 + 2) * U
    bad = np.abs(dp - dy * quotient) - np.abs(dy) * tol
    assert np.all(bad <= 0), (act, float(bad.max()))


@pytest.mark.parametrize("act,alpha", [("silu", 1.0), ("silu", 1.702), ("gelu", 1.0), ("gelu_tanh", 1.0)])
@pytest.mark.parametrize("M,N,ea", [(5, 40, "e2m1"), (300, 1000, "e2m1"), (300, 1000, "e4m3"), (1500, 2500, "e2m1"),
                                    (1500, 4000, "e4m3")])
def test_dense(act, alpha, M, N, ea):
    """One size for each of the layer's kernels: 16 rows, 128-row tiles, both pipelines."""
    need_gpu()
    banner(f"linear gradient against differences {M}x{N} {ea} {act}")
    rng = np.random.default_rng([M, N])
    K = 160
    qa, a = operand(rng, M, K, ea)
    qb, b = operand(rng, N, K, ea, std=1.5 / np.sqrt(K))
    bias = rng.standard_normal(N).astype(np.float32)
    dy = rng.standard_normal((M, N)).astype(np.float32)
    dp = host(mx.linear_backward(qa, qb, to_dev(dy), to_dev(bias), act, alpha=alpha, out_dtype=F32)).astype(np.float64)
    rows = np.unique(np.linspace(0, M - 1, 40).astype(int))
    P, err = projections(a[rows], b, ea == "e2m1")
    P = P + bias
    check_slope(dp[rows], dy[rows].astype(np.float64), P, err + U * np.abs(P), act, alpha)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("counts,N,ea", [([3, 0, 9], 48, "e2m1"), ([300, 0, 150], 1000, "e4m3"), ([1300, 0, 900], 2500, "e2m1"),
                                         ([1300, 0, 900], 2500, "e4m3")])
def test_grouped(act, counts, N, ea):
    need_gpu()
    banner(f"grouped linear gradient against differences {counts} {N} {ea} {act}")
    rng = np.random.default_rng([len(counts), N])
    K, M = 96, sum(counts)
    off, qa, a, qb, bs = grouped(rng, counts, M, N, K, ea, ea)
    bias = rng.standard_normal((len(counts), N)).astype(np.float32)
    dy = rng.standard_normal((M, N)).astype(np.float32)
    dp = host(mx.grouped_linear_backward(qa, to_dev(off), qb, to_dev(dy), to_dev(bias), act, out_dtype=F32)).astype(np.float64)
    for e, n in enumerate(counts):
        if n:
            rows = off[e] + np.unique(np.linspace(0, n - 1, 30).astype(int))
            P, err = projections(a[rows], bs[e], ea == "e2m1")
            P = P + bias[e]
            check_slope(dp[rows], dy[rows].astype(np.float64), P, err + U * np.abs(P), act, 1.0)
