"""The gated feed-forward block on MX operands (mx_gemm_gated and its backward
and grouped forms) against the formula in float64 on the oracle's dequantized
operands.

Tolerances follow from the arithmetic.  A projection is a float32 sum of n =
ceil(K / 64) matrix steps (each one rounding for FP4 operands) in at most 8
parts, so it errs by e = (n + 8) 2^-24 sum|a b|, plus the matrix instruction's
alignment allowance for FP8 / FP6.  The block is Lipschitz in the projections
(|act'| <= 1.13, |act''| <= 0.85 max(1, alpha), clamps 1), and evaluating it
costs a few float32 roundings, the exponential's growing with |z|; in the
derivative the error of 1 - s (2-3 of 2^-24) is multiplied by x z' <= 35 (the
tanh form where s is not yet 1).  bf16 outputs add half an ulp.  Where a projection is within e of the clamp, its
gradient may be either side's.
"""
import numpy as np
import pytest
import torch
from scipy.special import erf

import mxfp4_microscaling_quantization_mx_amd as mx
import oracle
from oracle.gemm import dequant_f64
from gpu_util import banner, bf16_half_ulp, host, mx_group_bound, need_gpu, to_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CLAMPED = mx.Gate("silu", 1.702, 7.0, 1.0)
# limits well inside the projections' spread, so that both sides of each clamp occur
TIGHT = mx.Gate("silu", 1.702, 1.25, 1.0)


def operand(rng, rows, K, elem="e2m1", block="1d", std=1.0, pad=16):
    """Oracle-quantized normal values: the MXTensor and its float64 values."""
    x = (rng.standard_normal((rows, K)) * std).astype(np.float32)
    codes, scales = oracle.quantize(x, block=block, elem=elem)
    buf = torch.full((scales.shape[0], max(1, -(-scales.shape[1] // pad) * pad)), 0xFF, dtype=torch.uint8,
                     device="cuda")
    buf[:, :scales.shape[1]] = to_dev(scales)
    cb = torch.zeros(rows, -(-codes.shape[1] // 16) * 16, dtype=torch.uint8, device="cuda")
    cb[:, :codes.shape[1]] = to_dev(codes)
    q = mx.MXTensor(cb[:, :codes.shape[1]], buf[:, :scales.shape[1]], rows, K, block, elem)
    return q, dequant_f64(codes, scales, elem, block)


def act(x, gate):
    """act(x), its derivative and the |z| of its exponential, in float64."""
    if gate.act == "gelu":
        cdf = 0.5 * (1 + erf(x / np.sqrt(2)))
        return x * cdf, cdf + x * np.exp(-0.5 * x * x) / np.sqrt(2 * np.pi), np.abs(x)
    if gate.act == "silu":
        z, dz = gate.alpha * x, gate.alpha
    else:
        c = 2 * np.sqrt(2 / np.pi)
        z, dz = c * (x + 0.044715 * x ** 3), c * (1 + 3 * 0.044715 * x * x)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-z))
    return x * s, s + x * s * (1 - s) * dz, np.abs(z)


def split(P, gate):
    N = P.shape[1] // 2
    return (P[:, 0::2], P[:, 1::2]) if gate.layout == "interleaved" else (P[:, :N], P[:, N:])


def join(dg, du, gate):
    if gate.layout == "halves":
        return np.concatenate([dg, du], 1)
    return np.stack([dg, du], -1).reshape(dg.shape[0], -1)


def projections(a, b, exact_products=True):
    """float64 P = a b^T and the float32 kernel's error bound on it."""
    n = -(-a.shape[1] // 64)
    e = (n + 8) * U * (np.abs(a) @ np.abs(b).T)
    if not exact_products:
        e = e + mx_group_bound(a, b)
    return a @ b.T, e


def check(out, ref, tol, bf16, alt=None, what=""):
    """|out - ref| <= tol (or |out - alt| <= tol where alt differs)."""
    out = np.asarray(out, dtype=np.float64)

    def miss(r):
        t = tol + (bf16_half_ulp(np.abs(r) + tol) if bf16 else 0.0)
        return np.abs(out - r) - t

    over = miss(ref)
    if alt is not None:
        over = np.minimum(over, miss(alt))
    assert np.isfinite(out).all(), what
    bad = over > 0
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst by {over.max():.3e}"


def forward_ref(P, eP, gate):
    (g, u), (eg, eu) = split(P, gate), split(eP, gate)
    lim = np.inf if gate.limit is None else gate.limit
    gc, v = np.minimum(g, lim), np.clip(u, -lim, lim) + gate.up_shift
    a, _, z = act(gc, gate)
    tol = 1.13 * np.abs(v) * eg + (np.abs(a) + 1.13 * eg) * eu + np.abs(a * v) * (16 + 2 * z) * U + 1e-37
    return a * v, tol + np.abs(a) * np.abs(gate.up_shift) * U + 4 * U * np.abs(gc * v)


def backward_ref(P, eP, dh, gate):
    """(dP, tolerance, the other side's dP where a projection is at a clamp)."""
    (g, u), (eg, eu) = split(P, gate), split(eP, gate)
    lim = np.inf if gate.limit is None else gate.limit
    gc, v = np.minimum(g, lim), np.clip(u, -lim, lim) + gate.up_shift
    a, d, z = act(gc, gate)
    dg, du = dh * v * d, dh * a
    tg = np.abs(dh) * (1.13 * eu + (np.abs(v) + eu) * 0.85 * max(1.0, gate.alpha) * eg) + np.abs(dh * v) * 128 * U
    tu = np.abs(dh) * (1.13 * eg + np.abs(a) * (16 + 2 * z) * U + 4 * U * np.abs(gc))
    og, ou = g > lim, np.abs(u) > lim
    ng, nu = np.abs(g - lim) <= eg, np.abs(np.abs(u) - lim) <= eu
    z = np.zeros_like(dg)
    ref = join(np.where(og, z, dg), np.where(ou, z, du), gate)
    alt = join(np.where(og != ng, z, dg), np.where(ou != nu, z, du), gate)
    return ref, join(tg, tu, gate) + 1e-37, alt


def run_case(M, N, K, gate, ea="e2m1", eb="e2m1", a_block="1d", b_block="1d", out=torch.float32, dh_dtype=None,
             pad=16, seed=0, b_std=None):
    rng = np.random.default_rng([seed, M, N, K])
    qa, a = operand(rng, M, K, ea, a_block, pad=pad)
    qb, b = operand(rng, 2 * N, K, eb, b_block, std=b_std or 1.5 / np.sqrt(K), pad=pad)
    banner(f"gated {M}x{N}x{K} {ea}/{eb} {a_block}/{b_block} {gate} {out}")
    P, e = projections(a, b, ea == eb == "e2m1")
    bf16 = out == torch.bfloat16
    # outputs inside a larger buffer: rows and columns around them stay untouched
    buf = torch.full((M + 2, N + 5), 3.0, dtype=out, device="cuda")
    mx.gemm_gated(qa, qb, gate, out=buf[1:M + 1, 2:N + 2])
    got = host(buf.float())
    ref, tol = forward_ref(P, e, gate)
    check(got[1:M + 1, 2:N + 2], ref, tol, bf16, what="h")
    got[1:M + 1, 2:N + 2] = 3.0
    assert np.all(got == 3.0), "written outside h"

    dh = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32)).to(dh_dtype or out)
    dhd = torch.full((M, N + 3), 7.0, dtype=dh.dtype, device="cuda")
    dhd[:, 1:N + 1] = dh.cuda()
    buf = torch.full((M + 2, 2 * N + 5), 3.0, dtype=out, device="cuda")
    mx.gemm_gated_backward(qa, qb, dhd[:, 1:N + 1], gate, out=buf[1:M + 1, 1:2 * N + 1])
    got = host(buf.float())
    ref, tol, alt = backward_ref(P, e, dh.double().numpy(), gate)
    check(got[1:M + 1, 1:2 * N + 1], ref, tol, bf16, alt, "dP")
    got[1:M + 1, 1:2 * N + 1] = 3.0
    assert np.all(got == 3.0), "written outside dP"


@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 2880, 2880), (3, 17, 64), (31, 16, 96), (32, 48, 2880),
                                   (33, 15, 416), (64, 33, 4128), (130, 129, 288), (300, 300, 160)])
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_shapes(M, N, K, layout, out):
    """One row to several tiles, widths that end inside a tile, K of one block
    to long, an odd block count; both layouts and output types."""
    need_gpu()
    run_case(M, N, K, mx.Gate("silu", 1.702, 7.0, 1.0, layout), out=out)


@pytest.mark.parametrize("gate", [mx.Gate(), mx.Gate("gelu"), mx.Gate("gelu_tanh"), CLAMPED, TIGHT,
                                  mx.Gate("gelu", limit=0.75, up_shift=-0.5), mx.Gate("gelu_tanh", limit=2.0)])
@pytest.mark.parametrize("std", [0.03, 0.5])
def test_activations(gate, std):
    """Every activation with and without clamps, at projections of a few units
    and far out in the activations' tails."""
    need_gpu()
    run_case(40, 50, 1024, gate, b_std=std)


ELEMS = ["e2m1", "e4m3", "e5m2", "e2m3", "e3m2"]


@pytest.mark.parametrize("ea", ELEMS)
@pytest.mark.parametrize("eb", ELEMS)
@pytest.mark.parametrize("M,N,K", [(5, 24, 96), (70, 40, 288)])
def test_element_types(ea, eb, M, N, K):
    """Every pair of element types (a K that ends inside a 64-deep step)."""
    need_gpu()
    run_case(M, N, K, CLAMPED, ea, eb)


@pytest.mark.parametrize("a_block,b_block", [("1d", "2d"), ("2d", "1d"), ("2d", "2d")])
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("M,N", [(64, 48), (288, 272), (512, 304)])
def test_two_dimensional_scales(a_block, b_block, layout, M, N):
    """2-D scales on either operand: gate and up rows of one column share a
    tile when interleaved and lie in different ones as halves."""
    need_gpu()
    run_case(M, N, 320, mx.Gate("silu", 1.702, 7.0, 1.0, layout), a_block=a_block, b_block=b_block)


@pytest.mark.parametrize("ea,eb", [("e2m1", "e2m1"), ("e4m3", "e4m3"), ("e2m3", "e5m2"), ("e2m1", "e4m3")])
@pytest.mark.parametrize("M,N,K", [(256, 128, 256), (257, 131, 288), (520, 300, 800), (300, 700, 2880),
                                   (1030, 257, 544)])
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_large_tiles(ea, eb, M, N, K, layout):
    """Shapes of whole and ragged 256-row tiles, K tails of 1 to 7 blocks."""
    need_gpu()
    run_case(M, N, K, mx.Gate("silu", 1.702, 1.25, 1.0, layout), ea, eb, out=torch.bfloat16, dh_dtype=torch.bfloat16)


@pytest.mark.parametrize("pad", [1, 4])
@pytest.mark.parametrize("ea,eb", [("e2m1", "e2m1"), ("e4m3", "e2m3")])
def test_scale_row_strides(pad, ea, eb):
    """Dense and 4-byte scale rows (no tile kernel takes them)."""
    need_gpu()
    run_case(300, 150, 2880, CLAMPED, ea, eb, pad=pad)


def test_mixed_output_and_gradient_types():
    need_gpu()
    run_case(37, 61, 160, CLAMPED, out=torch.float32, dh_dtype=torch.bfloat16)
    run_case(261, 161, 160, CLAMPED, out=torch.bfloat16, dh_dtype=torch.float32)


def _grouped(rng, counts, cap, E, N, K, eb="e2m1", ea="e2m1", b_block="2d"):
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    qa, a = operand(rng, cap, K, ea)
    parts = [operand(rng, 2 * N, K, eb, b_block, std=1.5 / np.sqrt(K)) for _ in range(E)]
    codes = torch.stack([p[0].codes._base for p in parts])[:, :, :parts[0][0].codes.shape[1]]
    scales = torch.stack([p[0].scales._base for p in parts])[:, :, :K // 32]
    qb = mx.MXTensor(codes, scales, 2 * N, K, b_block, eb)
    return off, qa, a, qb, [p[1] for p in parts]


@pytest.mark.parametrize("counts,N,K", [
    ([0, 1, 0, 2], 48, 96), ([33, 0, 31, 1, 100], 32, 64), ([700, 0, 3, 256, 257, 0], 160, 288),
    ([0, 0, 0], 16, 32), ([1] * 70, 16, 64), ([300, 20], 272, 800)])
@pytest.mark.parametrize("ea,eb", [("e2m1", "e2m1"), ("e4m3", "e4m3"), ("e4m3", "e2m1")])
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_grouped(counts, N, K, ea, eb, layout):
    """Experts without rows, with one and with several tiles, more than 64
    experts; rows past the last offset keep what was there."""
    need_gpu()
    rng = np.random.default_rng([7, len(counts), N, K])
    gate, E, total = mx.Gate("silu", 1.702, 1.25, 1.0, layout), len(counts), int(np.sum(counts))
    cap = total + 5
    off, qa, a, qb, bs = _grouped(rng, counts, cap, E, N, K, eb, ea)
    banner(f"grouped gated {counts} {N}x{K} {ea}/{eb} {layout}")
    offd = to_dev(off)
    H = torch.full((cap, N), 3.0, device="cuda")
    mx.grouped_gemm_gated(qa, offd, qb, gate, out=H)
    dh = rng.standard_normal((cap, N)).astype(np.float32)
    dP = torch.full((cap, 2 * N), 3.0, device="cuda")
    mx.grouped_gemm_gated_backward(qa, offd, qb, to_dev(dh), gate, out=dP)
    H, dP = host(H), host(dP)
    assert np.all(H[total:] == 3.0) and np.all(dP[total:] == 3.0)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        P, err = projections(a[lo:hi], bs[e], ea == eb == "e2m1")
        ref, tol = forward_ref(P, err, gate)
        check(H[lo:hi], ref, tol, False, what=f"h of expert {e}")
        ref, tol, alt = backward_ref(P, err, dh[lo:hi].astype(np.float64), gate)
        check(dP[lo:hi], ref, tol, False, alt, f"dP of expert {e}")


def test_grouped_offsets_are_clamped():
    """Offsets past the capacity are clamped to it, negative ones to 0."""
    need_gpu()
    rng = np.random.default_rng(3)
    _, qa, a, qb, bs = _grouped(rng, [20, 20], 40, 2, 16, 64)
    banner("grouped gated, offsets out of range")
    H = host(mx.grouped_gemm_gated(qa, to_dev(np.array([-5, 20, 1000], dtype=np.int32)), qb, CLAMPED, torch.float32))
    for e, (lo, hi) in enumerate([(0, 20), (20, 40)]):
        ref, tol = forward_ref(*projections(a[lo:hi], bs[e]), CLAMPED)
        check(H[lo:hi], ref, tol, False)


def test_more_experts_than_the_pipelines_table():
    """1000 experts, some empty, 8300 rows: past the tile pipelines' table."""
    need_gpu()
    rng = np.random.default_rng(21)
    counts = rng.integers(0, 18, 1000)
    counts[-1] += max(0, 8300 - counts.sum())
    off, qa, a, qb, bs = _grouped(rng, counts, int(counts.sum()), 1000, 64, 64)
    banner("grouped gated 1000 experts")
    H = host(mx.grouped_gemm_gated(qa, to_dev(off), qb, CLAMPED, torch.float32))
    for e in list(range(0, 1000, 37)) + [999]:
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            ref, tol = forward_ref(*projections(a[lo:hi], bs[e]), CLAMPED)
            check(H[lo:hi], ref, tol, False, what=f"expert {e}")


@pytest.mark.parametrize("M", [3, 200, 1100])
def test_graph_replays_equal_eager_calls(M):
    """A captured forward and backward pass, replayed between eager calls on
    changing inputs."""
    need_gpu()
    rng = np.random.default_rng(31)
    qb, _ = operand(rng, 2 * 272, 288, std=0.1)
    inputs = [operand(rng, M, 288)[0] for _ in range(3)]
    qa = operand(rng, M, 288)[0]
    dh = torch.randn(M, 272, device="cuda")
    run = lambda q: (mx.gemm_gated(q, qb, CLAMPED, torch.float32),
                     mx.gemm_gated_backward(q, qb, dh, CLAMPED, torch.float32))
    banner(f"gated graph M={M}")
    run(qa)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(qa)
    for q in inputs:
        qa.codes.copy_(q.codes)
        qa.scales.copy_(q.scales)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, run(q)))


@pytest.mark.parametrize("M,N", [(20, 24), (300, 160)])
def test_nan_scales_poison_their_outputs_only(M, N):
    """A NaN scale of an A row makes that row NaN, one of a gate or up row its
    column; everything else is untouched, clamps included (a clamp keeps NaN)."""
    need_gpu()
    rng = np.random.default_rng(5)
    qa, a = operand(rng, M, 160)
    qb, b = operand(rng, 2 * N, 160, std=0.1)
    qa.scales[2, 3] = 0xFF
    qb.scales[2 * 4, 0] = 0xFF                       # gate of column 4
    qb.scales[2 * 9 + 1, 4] = 0xFF                   # up of column 9
    banner(f"gated NaN scales {M}x{N}")
    h = host(mx.gemm_gated(qa, qb, TIGHT, torch.float32))
    dP = host(mx.gemm_gated_backward(qa, qb, torch.ones(M, N, device="cuda"), TIGHT, torch.float32))
    want = np.zeros((M, N), bool)
    want[2], want[:, 4], want[:, 9] = True, True, True
    assert np.array_equal(np.isnan(h), want)
    rows = np.arange(M) != 2
    assert np.isnan(dP[rows][:, 2 * 4]).all() and not np.isnan(dP[rows][:, 16]).any()
    ok = np.ones(2 * N, bool)
    ok[[8, 9, 18, 19]] = False
    assert not np.isnan(dP[rows][:, ok]).any()


def test_empty_and_zero():
    """M = 0 and N = 0 write nothing; K = 0 projects to zero; zero operands too."""
    need_gpu()
    banner("gated empty")
    e = lambda r, k: mx.MXTensor(torch.zeros(r, max(16, k // 2), dtype=torch.uint8, device="cuda"),
                                 torch.zeros(r, max(1, k // 32), dtype=torch.uint8, device="cuda"), r, k)
    assert mx.gemm_gated(e(0, 64), e(32, 64)).shape == (0, 16)
    assert mx.gemm_gated(e(3, 64), e(0, 64)).shape == (3, 0)
    for M, N in ((3, 5), (300, 160)):
        for K in (0, 64):
            gate = mx.Gate(up_shift=2.0)
            assert np.all(host(mx.gemm_gated(e(M, K), e(2 * N, K), gate, torch.float32)) == 0.0)
            dP = host(mx.gemm_gated_backward(e(M, K), e(2 * N, K), torch.ones(M, N, device="cuda"), gate,
                                             torch.float32))
            assert np.all(dP[:, 0::2] == 1.0) and np.all(dP[:, 1::2] == 0.0)   # 2 * silu'(0), silu(0)


@pytest.mark.parametrize("gate", [mx.Gate(), mx.Gate("gelu"), mx.Gate("gelu_tanh"), CLAMPED])
def test_extreme_projections(gate):
    """Projections from 1e-30 to 1e30 of either sign: no overflow of the
    exponential or of a polynomial reaches the result."""
    need_gpu()
    mags = np.array([1e-30, 1e-8, 1.0, 8.0, 20.0, 100.0, 1e4, 1e12, 1e18])
    vals = np.concatenate([mags, -mags])
    n = len(vals)
    # a = one 1.0 per row, b = the value to the nearest power of two as a scale
    e = np.round(np.log2(np.abs(vals))).astype(int)
    vals = np.sign(vals) * 2.0 ** e
    ac = np.zeros((1, 16), np.uint8)
    ac[0, 0] = 2
    rows, scales = [], []
    for x, k in zip(vals, e):
        for r in (x, 1.0):
            c = np.zeros(16, np.uint8)
            c[0] = 2 | (8 if r < 0 else 0)
            rows.append(c)
            scales.append([127 + (k if r is x else 0)])
    qa = mx.MXTensor(to_dev(ac), to_dev(np.full((1, 1), 127, np.uint8)), 1, 32)
    qb = mx.MXTensor(to_dev(np.stack(rows)), to_dev(np.array(scales, np.uint8)), 2 * n, 32)
    banner(f"gated extremes {gate}")
    P = np.stack([vals, np.ones(n)], -1).reshape(1, -1)
    h = host(mx.gemm_gated(qa, qb, gate, torch.float32))
    ref, tol = forward_ref(P, np.zeros_like(P), gate)
    check(h, ref, np.where(np.abs(ref) < 1e-30, 1e-30, tol), False)
    dP = host(mx.gemm_gated_backward(qa, qb, torch.ones(1, n, device="cuda"), gate, torch.float32))
    ref, tol, _ = backward_ref(P, np.zeros_like(P), np.ones((1, n)), gate)
    check(dP, ref, np.maximum(tol, 1e-30), False)


@pytest.mark.parametrize("gate", [mx.Gate(), mx.Gate("gelu"), mx.Gate("gelu_tanh"), CLAMPED])
def test_backward_against_differences(gate):
    """dP against central differences of the forward formula in float64 (the
    formula of the test's own derivative is checked on the way)."""
    need_gpu()
    rng = np.random.default_rng(11)
    qa, a = operand(rng, 24, 128)
    qb, b = operand(rng, 2 * 20, 128, std=0.12)
    P = a @ b.T
    dh = rng.standard_normal((24, 20)).astype(np.float32)
    banner(f"gated differences {gate}")
    got = host(mx.gemm_gated_backward(qa, qb, to_dev(dh), gate, torch.float32))
    eps, z = 1e-5, np.zeros_like(P)
    num = np.zeros_like(P)
    for c in range(P.shape[1]):
        d = z.copy()
        d[:, c] = eps
        hp, hm = forward_ref(P + d, z, gate)[0], forward_ref(P - d, z, gate)[0]
        num[:, c] = ((hp - hm) / (2 * eps) * dh).sum(1)
    near = np.abs(np.abs(P) - (np.inf if gate.limit is None else gate.limit)) < 1e-4
    # differences err by eps^2 / 6 of the third derivative and 1e-16 / eps of rounding
    assert np.abs(np.where(near, 0, got - num)).max() < 1e-4 * max(1.0, np.abs(num).max())


def test_same_bits_every_run_and_other_stream():
    """The sums have a fixed order: equal bits from run to run, and from
    another stream once that stream has waited for the inputs."""
    need_gpu()
    rng = np.random.default_rng(13)
    qa, _ = operand(rng, 300, 2880)
    qb, _ = operand(rng, 320, 2880, std=0.02)
    banner("gated repeat")
    one = mx.gemm_gated(qa, qb, CLAMPED, torch.float32)
    two = mx.gemm_gated(qa, qb, CLAMPED, torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        three = mx.gemm_gated(qa, qb, CLAMPED, torch.float32)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(one, two) and torch.equal(one, three)


@pytest.mark.parametrize("backward", [False, True])
def test_full_size_sampled_rows(backward):
    """16384 x 2880 x 2880 with 2-D weight tiles (quantized on the GPU from
    seeded normals), 96 sampled rows against float64 on all columns."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(17)
    x = torch.randn(16384, 2880, device="cuda", generator=g).to(torch.bfloat16)
    w = (torch.randn(5760, 2880, device="cuda", generator=g) * 0.02).to(torch.bfloat16)
    qa, qb = mx.quantize(x), mx.quantize(w, block="2d")
    dh = (torch.randn(16384, 2880, device="cuda", generator=g) * 1e-3).to(torch.bfloat16)
    banner(f"gated full size backward={backward}")
    rows = np.sort(np.random.default_rng(1).choice(16384, 96, replace=False))
    rows[[0, -1]] = 0, 16383
    out = mx.gemm_gated_backward(qa, qb, dh, CLAMPED) if backward else mx.gemm_gated(qa, qb, CLAMPED)
    got = host(out[torch.from_numpy(rows).cuda()].float())
    a = host(mx.dequantize(qa)[torch.from_numpy(rows).cuda()]).astype(np.float64)
    b = host(mx.dequantize(qb)).astype(np.float64)
    P, e = projections(a, b)
    if backward:
        d = dh[torch.from_numpy(rows).cuda()].double().cpu().numpy()
        ref, tol, alt = backward_ref(P, e, d, CLAMPED)
        check(got, ref, tol, True, alt)
    else:
        ref, tol = forward_ref(P, e, CLAMPED)
        check(got, ref, tol, True)
