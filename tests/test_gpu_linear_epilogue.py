"""The linear layer with bias, activation and residual in its epilogue (mx_linear, its
backward and grouped forms) against the formula in float64 on the oracle's
dequantized operands.

Tolerances follow from the arithmetic, with test_gpu_gated's bound e on the sum of
products.  Adding the bias rounds once: x errs by ex = e + 2^-24 (|x| + e).  The
activations are Lipschitz (|act'| <= 1.13, |act''| <= 0.85 max(1, alpha)) and err by
(16 + 2 |z| + 1.25 x^2) 2^-24 of themselves, their derivatives by 128 of 2^-24;
adding the residual and multiplying by dy round once more, then the output's type.
"""
import numpy as np
import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx
from gpu_util import banner, host, need_gpu, to_dev
from test_gpu_gated import ELEMS, U, act, check, operand, projections

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ACTS = [None, "silu", "gelu", "gelu_tanh"]


def value_ref(P, e, bias, name, alpha, r):
    """(Y, tolerance)."""
    x = P if bias is None else P + bias
    ex = e + U * (np.abs(x) + e)
    if name is None:
        y, tol = x, ex
    else:
        y, _, z = act(x, mx.Gate(name, alpha))
        tol = 1.13 * ex + np.abs(y) * (16 + 2 * z + 1.25 * x * x * (name == "gelu")) * U
    if r is not None:
        y = y + r
        tol = tol + U * (np.abs(y) + tol)
    return y, tol + 1e-37


def gradient_ref(P, e, bias, name, alpha, dy):
    x = P if bias is None else P + bias
    ex = e + U * (np.abs(x) + e)
    _, d, _ = act(x, mx.Gate(name, alpha))
    return dy * d, np.abs(dy) * (0.85 * max(1.0, alpha) * ex + 128 * U) + 1e-37


def framed(M, N, dtype, rng=None, pad=5, at=2):
    """A [M, N] view inside a larger buffer of 3s, with normal values if rng."""
    buf = torch.full((M + 2, N + pad), 3.0, dtype=dtype, device="cuda")
    t = buf[1:M + 1, at:N + at]
    if rng is not None:
        t.copy_(to_dev(rng.standard_normal((M, N)).astype(np.float32)).to(dtype))
    return buf, t


def untouched(buf, t, at=2):
    got = buf.clone()
    got[1:t.shape[0] + 1, at:t.shape[1] + at] = 3.0
    assert bool((got == 3.0).all()), "written outside the output"


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def sample_rows(M, N):
    """All rows, or those at the borders of tiles and some between."""
    if M * N <= 600_000:
        return np.arange(M)
    edge = [r for c in range(0, M + 128, 128) for r in (c - 1, c, c + 33) if 0 <= r < M]
    return np.unique(np.array(edge + [M - 1]))


def run_case(M, N, K, name, ea="e2m1", eb="e2m1", a_block="1d", b_block="1d", out=F32, bias=F32, res=F32, alpha=1.0,
             scale_pad=16, pad=5, at=2, b_std=None, seed=0):
    rng = np.random.default_rng([seed, M, N, K])
    qa, a = operand(rng, M, K, ea, a_block, pad=scale_pad)
    qb, b = operand(rng, N, K, eb, b_block, std=b_std or 1.5 / np.sqrt(max(K, 1)), pad=scale_pad)
    banner(f"linear {M}x{N}x{K} {ea}/{eb} {a_block}/{b_block} {name} {out} {bias} {res}")
    rows = sample_rows(M, N)
    P, e = projections(a[rows], b, ea == eb == "e2m1")
    bt = None if bias is None else to_dev(rng.standard_normal(N).astype(np.float32)).to(bias)
    r = None if res is None else framed(M, N, res, rng, pad, at)[1]
    rr = None if r is None else f64(r)[rows]
    buf, y = framed(M, N, out, pad=pad, at=at)
    mx.linear(qa, qb, bt, name, r, alpha, out=y)
    ref, tol = value_ref(P, e, f64(bt), name, alpha, rr)
    check(host(y.float())[rows], ref, tol, out == BF16, what="y")
    untouched(buf, y, at)
    if name is None:
        return
    dy = framed(M, N, res or out, rng, pad, at)[1]
    buf, dp = framed(M, N, out, pad=pad, at=at)
    mx.linear_backward(qa, qb, dy, bt, name, alpha, out=dp)
    ref, tol = gradient_ref(P, e, f64(bt), name, alpha, f64(dy)[rows])
    check(host(dp.float())[rows], ref, tol, out == BF16, what="dp")
    untouched(buf, dp, at)


@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 2880, 2880), (3, 17, 64), (31, 32, 96), (32, 48, 2880), (33, 31, 416),
                                   (64, 33, 4128), (130, 129, 288), (300, 300, 160)])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("out", [F32, BF16])
def test_shapes(M, N, K, name, out):
    """One row to several tiles, widths that end inside a tile, K of one block to
    long, an odd block count."""
    need_gpu()
    run_case(M, N, K, name, out=out, bias=out, res=out)


@pytest.mark.parametrize("bias", [None, F32, BF16])
@pytest.mark.parametrize("res", [None, F32, BF16])
@pytest.mark.parametrize("M,N", [(40, 50), (420, 1800), (1100, 3801)])
def test_bias_and_residual_types(bias, res, M, N):
    """Each with and without, at every kernel, in types of their own."""
    need_gpu()
    for name in (None, "silu"):
        run_case(M, N, 96, name, bias=bias, res=res, out=BF16)
        run_case(M, N, 96, name, bias=bias, res=res, out=F32, pad=0, at=0)


@pytest.mark.parametrize("pad,at", [(0, 0), (1, 0), (2, 2), (6, 1), (3, 0)])
@pytest.mark.parametrize("ea", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,N", [(1100, 3840), (1100, 3842), (1100, 3839)])
def test_buffer_strides_of_the_pipelines(pad, at, ea, M, N):
    """Rows that whole bf16 lines fit, and those that start at odd elements."""
    need_gpu()
    N = N if ea == "e2m1" else N + 3584                  # (past the tile kernel's range)
    run_case(M, N, 64, "gelu_tanh", ea, ea, out=BF16, bias=BF16, res=BF16, pad=pad, at=at)


@pytest.mark.parametrize("ea", ELEMS)
@pytest.mark.parametrize("eb", ELEMS)
@pytest.mark.parametrize("M,N,K", [(5, 48, 96), (70, 40, 288), (420, 1800, 288)])
def test_element_types(ea, eb, M, N, K):
    """Every pair of element types (a K that ends inside a 64-deep step)."""
    need_gpu()
    run_case(M, N, K, "silu", ea, eb, alpha=1.702)


@pytest.mark.parametrize("a_block,b_block", [("1d", "2d"), ("2d", "1d"), ("2d", "2d")])
@pytest.mark.parametrize("elem,M,N", [("e2m1", 64, 96), ("e2m1", 448, 1824), ("e4m3", 448, 1824), ("e2m1", 1120, 3808),
                                      ("e4m3", 1120, 7424)])
def test_two_dimensional_scales(a_block, b_block, elem, M, N):
    need_gpu()
    run_case(M, N, 160, "gelu", elem, elem, a_block, b_block)


@pytest.mark.parametrize("a_block", ["1d", "2d"])
@pytest.mark.parametrize("bias", [F32, BF16])
@pytest.mark.parametrize("N", [3840, 3842, 3841, 3585])
def test_bias_of_long_products(a_block, bias, N):
    """Tiles of enough stages that their bias is brought to LDS beside them: widths that
    end at and inside a tile, at an odd column; a bias row that starts at an odd element."""
    need_gpu()
    rng = np.random.default_rng([N, 3])
    M, K = 1088, 832
    qa, a = operand(rng, M, K, block=a_block)
    qb, b = operand(rng, N, K, std=0.05)
    rows = np.array([0, 31, 255, 256, 700, 1023, 1024, 1087])
    P, e = projections(a[rows], b)
    for shift in (0, 1, 2):
        banner(f"linear bias of long products {a_block} {bias} N={N} shift={shift}")
        bt = torch.full((N + 4,), 100.0, dtype=bias, device="cuda")[shift:shift + N]
        bt.copy_(to_dev(rng.standard_normal(N).astype(np.float32)))
        for name in (None, "silu"):
            ref, tol = value_ref(P, e, f64(bt), name, 1.0, None)
            check(host(mx.linear(qa, qb, bt, name, out_dtype=F32))[rows], ref, tol, False)


@pytest.mark.parametrize("bias", [F32, BF16])
def test_grouped_bias_of_long_products(bias):
    """The same per expert, bias rows a stride apart that starts them at odd elements."""
    need_gpu()
    rng = np.random.default_rng(17)
    counts, N, K = [1300, 0, 900, 77], 2401, 640
    off, qa, a, qb, bs = grouped(rng, counts, sum(counts), N, K)
    for stride in (2401, 2402, 2404):
        banner(f"grouped linear bias of long products {bias} stride={stride}")
        bt = torch.zeros(4, stride, dtype=bias, device="cuda")[:, :N]
        bt.copy_(to_dev(rng.standard_normal((4, N)).astype(np.float32)))
        y = host(mx.grouped_linear(qa, to_dev(off), qb, bt, out_dtype=F32))
        check_groups(off, a, bs, f64(bt), None, None, y, None, None, True)


@pytest.mark.parametrize("elem,M,N", [("e2m1", 1120, 3808), ("e4m3", 1120, 7424)])
@pytest.mark.parametrize("b_block", ["1d", "2d"])
def test_two_dimensional_scales_without_an_activation(elem, M, N, b_block):
    need_gpu()
    run_case(M, N, 608, None, elem, elem, "2d", b_block, out=BF16, res=BF16)


@pytest.mark.parametrize("scale_pad", [1, 2, 4])
@pytest.mark.parametrize("ea,eb", [("e2m1", "e2m1"), ("e4m3", "e4m3"), ("e4m3", "e2m3")])
@pytest.mark.parametrize("M,N,K", [(40, 60, 608), (420, 1800, 608), (1100, 3800, 288)])
def test_scale_row_strides(scale_pad, ea, eb, M, N, K):
    """Scale rows that start at any byte, or 4-byte ones."""
    need_gpu()
    run_case(M, N, K, "silu", ea, eb, scale_pad=scale_pad)


@pytest.mark.parametrize("ea,eb", [("e2m1", "e2m1"), ("e4m3", "e5m2"), ("e2m3", "e3m2"), ("e3m2", "e2m1")])
@pytest.mark.parametrize("M,N,K", [(400, 1920, 32), (513, 1667, 96), (897, 897, 128), (417, 1793, 480), (512, 1600, 544)])
def test_tile_depths(ea, eb, M, N, K):
    """One stage, fewer stages than the ring has slots, whole and partial last
    stages; rows and columns that end 1 into a tile and at its end."""
    need_gpu()
    run_case(M, N, K, "gelu_tanh", ea, eb)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("ea,eb,M,N,K", [
    ("e2m1", "e2m1", 1100, 3800, 96), ("e2m1", "e2m1", 1537, 2602, 256), ("e2m1", "e2m1", 1025, 3713, 544),
    ("e2m1", "e2m1", 1024, 4096, 800), ("e4m3", "e5m2", 1100, 7400, 96), ("e4m3", "e4m3", 1537, 5200, 256),
    ("e2m3", "e4m3", 1025, 7425, 288), ("e3m2", "e3m2", 1025, 7425, 544), ("e2m1", "e4m3", 1025, 3713, 288)])
def test_pipelines(name, ea, eb, M, N, K):
    """Ragged rows and columns and K tails of the 256-row pipelines (a mixed MXFP4
    pair keeps to 128 x 128 tiles)."""
    need_gpu()
    run_case(M, N, K, name, ea, eb, out=BF16, res=BF16)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("std", [0.03, 0.5])
def test_activations_far_out(name, std):
    need_gpu()
    run_case(40, 50, 1024, name, b_std=std)


@pytest.mark.parametrize("M,N", [(7, 40), (420, 1800), (1100, 3800)])
def test_no_products(M, N):
    """K = 0: act(bias) + residual."""
    need_gpu()
    banner(f"linear K=0 {M}x{N}")
    rng = np.random.default_rng(1)
    q = lambda rows: mx.MXTensor(torch.empty(rows, 0, dtype=torch.uint8, device="cuda"),
                                 torch.empty(rows, 0, dtype=torch.uint8, device="cuda"), rows, 0)
    bias, r = to_dev(rng.standard_normal(N).astype(np.float32)), to_dev(rng.standard_normal((M, N)).astype(np.float32))
    y = host(mx.linear(q(M), q(N), bias, "silu", r, out_dtype=F32))
    ref, tol = value_ref(np.zeros((M, N)), np.zeros((M, N)), f64(bias), "silu", 1.0, f64(r))
    check(y, ref, tol, False)


def test_empty_shapes():
    need_gpu()
    banner("linear without rows or columns")
    rng = np.random.default_rng(1)
    q, _ = operand(rng, 5, 64)
    none = mx.MXTensor(torch.empty(0, 32, dtype=torch.uint8, device="cuda"), torch.empty(0, 2, dtype=torch.uint8, device="cuda"),
                       0, 64)
    assert mx.linear(none, q).shape == (0, 5) and mx.linear(q, none).shape == (5, 0)
    assert mx.linear_backward(none, q, torch.empty(0, 5, device="cuda")).shape == (0, 5)


@pytest.mark.parametrize("M,N", [(7, 40), (420, 1800), (1100, 3800)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place(M, N, dtype):
    """Y over the residual, dP over dY."""
    need_gpu()
    banner(f"linear in place {M}x{N} {dtype}")
    rng = np.random.default_rng(4)
    qa, _ = operand(rng, M, 160)
    qb, _ = operand(rng, N, 160, std=0.1)
    for at in (0, 1):
        buf, r = framed(M, N, dtype, rng, 4, at)
        want = mx.linear(qa, qb, None, "silu", r.clone(), out_dtype=dtype)
        mx.linear(qa, qb, None, "silu", r, out=r)
        assert torch.equal(r, want)
        untouched(buf, r, at)
        buf, g = framed(M, N, dtype, rng, 4, at)
        want = mx.linear_backward(qa, qb, g.clone(), None, "gelu", out_dtype=dtype)
        mx.linear_backward(qa, qb, g, None, "gelu", out=g)
        assert torch.equal(g, want)


# ------------------------------------------------------------------ grouped
def grouped(rng, counts, cap, N, K, ea="e2m1", eb="e2m1", b_block="1d"):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    qa, a = operand(rng, cap, K, ea)
    parts = [operand(rng, N, K, eb, b_block, std=1.5 / np.sqrt(K)) for _ in counts]
    codes = torch.stack([p[0].codes._base for p in parts])[:, :, :parts[0][0].codes.shape[1]]
    scales = torch.stack([p[0].scales._base for p in parts])[:, :, :K // 32]
    return off, qa, a, mx.MXTensor(codes, scales, N, K, b_block, eb), [p[1] for p in parts]


def check_groups(off, a, bs, bias, r, dy, y, dp, name, exact, experts=None):
    for e in experts or range(len(bs)):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        rows = lo + sample_rows(hi - lo, bs[e].shape[0])
        P, err = projections(a[rows], bs[e], exact)
        be = None if bias is None else bias[e]
        ref, tol = value_ref(P, err, be, name, 1.0, None if r is None else r[rows])
        check(y[rows], ref, tol, False, what=f"y of expert {e}")
        if dp is not None:
            ref, tol = gradient_ref(P, err, be, name, 1.0, dy[rows])
            check(dp[rows], ref, tol, False, what=f"dp of expert {e}")


@pytest.mark.parametrize("counts,N,K", [
    ([0, 1, 0, 2], 48, 96), ([33, 0, 31, 1, 100], 32, 64), ([700, 0, 3, 256, 257, 0], 1184, 288), ([0, 0, 0], 16, 32),
    ([1] * 70, 16, 64), ([300, 20], 544, 800), ([1200, 0, 900], 1600, 96), ([1300, 0, 900, 77], 2400, 608),
    ([513, 800], 3872, 96)])
@pytest.mark.parametrize("ea,eb", [("e2m1", "e2m1"), ("e4m3", "e4m3"), ("e4m3", "e2m1")])
@pytest.mark.parametrize("b_block", ["1d", "2d"])
def test_grouped(counts, N, K, ea, eb, b_block):
    """Experts without rows, with one and with several tiles, more than 64 experts;
    rows past the last offset keep what was there."""
    need_gpu()
    if b_block == "2d" and N % 32:
        N = 32
    rng = np.random.default_rng([7, len(counts), N, K])
    E, total = len(counts), int(np.sum(counts))
    cap = total + 5
    off, qa, a, qb, bs = grouped(rng, counts, cap, N, K, ea, eb, b_block)
    banner(f"grouped linear {counts[:8]} {N}x{K} {ea}/{eb} {b_block}")
    offd, name = to_dev(off), "gelu_tanh"
    bias = torch.zeros(E, N + 3, device="cuda")[:, 1:N + 1]                # rows with a stride of their own
    bias.copy_(to_dev(rng.standard_normal((E, N)).astype(np.float32)))
    r = to_dev(rng.standard_normal((cap, N)).astype(np.float32))
    y = torch.full((cap, N), 3.0, device="cuda")
    mx.grouped_linear(qa, offd, qb, bias, name, r, out=y)
    dp = torch.full((cap, N), 3.0, device="cuda")
    mx.grouped_linear_backward(qa, offd, qb, r, bias, name, out=dp)
    y, dp = host(y), host(dp)
    assert np.all(y[total:] == 3.0) and np.all(dp[total:] == 3.0)
    check_groups(off, a, bs, f64(bias), f64(r), f64(r), y, dp, name, ea == eb == "e2m1")
    y = host(mx.grouped_linear(qa, offd, qb, out_dtype=F32))
    check_groups(off, a, bs, None, None, None, y, None, None, ea == eb == "e2m1")


def test_grouped_offsets_are_clamped():
    """Offsets past the capacity are clamped to it, negative ones to 0."""
    need_gpu()
    rng = np.random.default_rng(3)
    _, qa, a, qb, bs = grouped(rng, [20, 20], 40, 32, 64)
    banner("grouped linear, offsets out of range")
    bias = torch.randn(2, 32, device="cuda")
    y = host(mx.grouped_linear(qa, to_dev(np.array([-5, 20, 1000], dtype=np.int32)), qb, bias, out_dtype=F32))
    check_groups([0, 20, 40], a, bs, f64(bias), None, None, y, None, None, True)


def test_more_experts_than_the_pipelines_table():
    need_gpu()
    rng = np.random.default_rng(21)
    counts = rng.integers(0, 18, 1000)
    counts[-1] += max(0, 8300 - counts.sum())
    off, qa, a, qb, bs = grouped(rng, counts, int(counts.sum()), 64, 64)
    banner("grouped linear 1000 experts")
    bias = torch.randn(1000, 64, device="cuda").to(BF16)
    y = host(mx.grouped_linear(qa, to_dev(off), qb, bias, "silu", out_dtype=F32))
    check_groups(off, a, bs, f64(bias), None, None, y, None, "silu", True, list(range(0, 1000, 37)) + [999])


@pytest.mark.parametrize("M,N", [(3, 272), (200, 1900), (1100, 3800)])
def test_graph_replays_equal_eager_calls(M, N):
    """A captured forward and backward pass, replayed between eager calls on changing
    inputs, and the same on another stream."""
    need_gpu()
    rng = np.random.default_rng(31)
    qb, _ = operand(rng, N, 288, std=0.1)
    inputs = [operand(rng, M, 288)[0] for _ in range(3)]
    qa = operand(rng, M, 288)[0]
    bias, r = torch.randn(N, device="cuda"), torch.randn(M, N, device="cuda")
    run = lambda q: (mx.linear(q, qb, bias, "silu", r), mx.linear_backward(q, qb, r, bias, "gelu_tanh"))
    banner(f"linear graph M={M}")
    run(qa)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(qa)
    for q in inputs:
        qa.codes.copy_(q.codes)
        qa.scales.copy_(q.scales)
        r.add_(0.25)
        g.replay()
        torch.cuda.synchronize()
        want = run(q)
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = run(inputs[-1])
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(other, want))


@pytest.mark.parametrize("M,N", [(20, 48), (420, 1800), (1100, 3800)])
def test_nan_scales_poison_their_outputs_only(M, N):
    need_gpu()
    rng = np.random.default_rng(5)
    qa, _ = operand(rng, M, 160)
    qb, _ = operand(rng, N, 160, std=0.1)
    qa.scales[2, 3] = 0xFF
    qb.scales[8, 0] = 0xFF
    banner(f"linear NaN scales {M}x{N}")
    want = np.zeros((M, N), bool)
    want[2], want[:, 8] = True, True
    bias, r = torch.randn(N, device="cuda"), torch.randn(M, N, device="cuda")
    for name in ACTS:
        assert np.array_equal(np.isnan(host(mx.linear(qa, qb, bias, name, r, out_dtype=F32))), want)
        if name:
            assert np.array_equal(np.isnan(host(mx.linear_backward(qa, qb, r, bias, name, out_dtype=F32))), want)


def test_equal_to_the_product():
    """Without an epilogue, MXFP4 at a shape that mx_gemm does not split: its bits."""
    need_gpu()
    banner("linear against gemm")
    rng = np.random.default_rng(6)
    qa, _ = operand(rng, 4200, 320)
    qb, _ = operand(rng, 4100, 320)
    for dt in (F32, BF16):
        assert torch.equal(mx.linear(qa, qb, out_dtype=dt), mx.gemm(qa, qb, dt))


def test_outputs_past_32_bits():
    """4.4 GB of output and of residual: addresses past 32 bits."""
    need_gpu()
    M, N, K = 270000, 8192, 32
    banner(f"linear {M}x{N}x{K}")
    rng = np.random.default_rng(8)
    qa, a = operand(rng, M, K)
    qb, b = operand(rng, N, K)
    bias = torch.randn(N, device="cuda")
    r = torch.zeros(M, N, dtype=BF16, device="cuda")
    rows = np.array([0, 1, 131071, 131072, 262143, 262144, 269999])
    idx = torch.from_numpy(rows).cuda()
    r[idx] = torch.randn(rows.size, N, device="cuda").to(BF16)
    want = f64(r[idx])
    mx.linear(qa, qb, bias, None, r, out=r)              # in place
    P, e = projections(a[rows], b)
    ref, tol = value_ref(P, e, f64(bias), None, 1.0, want)
    check(host(r[idx].float()), ref, tol, True)
