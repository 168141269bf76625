"""What every kernel of the gated block has to do alike, run on each of them:
the kernel for few rows (K split over 8 or 2 waves), the 128 x 64 tiles, and
the 256-row pipelines of MXFP4 and of MXFP8 / MXFP6.  The sizes select them on
256 CUs: few rows up to 768 tiles of 32 x 16 (MXFP4; 640 wider), 128 x 64 tiles
up to 256 (512), pipelines above; grouped, few rows up to 8 rows per expert or
1536 tiles, pipelines above, and 128 x 64 tiles for what no pipeline takes."""
import numpy as np
import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx
from gpu_util import banner, host, need_gpu, to_dev
from test_gpu_gated import (CLAMPED, TIGHT, _grouped, backward_ref, check, forward_ref, operand, projections)

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TIGHT_HALVES = mx.Gate("silu", 1.702, 1.25, 1.0, "halves")
# element types of A and B, rows, hidden columns
PATHS = {
    "few, 8 waves": ("e2m1", "e2m1", 20, 24),
    "few, 2 waves": ("e2m1", "e2m1", 100, 2881),
    "tiles, mixed, one row of tiles": ("e4m3", "e2m1", 100, 2881),
    "tiles, MXFP4": ("e2m1", "e2m1", 420, 900),
    "tiles, MXFP8": ("e4m3", "e4m3", 420, 900),
    "tiles, mixed": ("e4m3", "e2m1", 420, 900),
    "tiles, MXFP6": ("e2m3", "e3m2", 420, 900),
    "pipeline, MXFP4": ("e2m1", "e2m1", 1100, 1900),
    "pipeline, MXFP8": ("e4m3", "e5m2", 1100, 3700),
    "pipeline, MXFP6": ("e2m3", "e2m3", 1100, 3700),
}
paths = pytest.mark.parametrize("path", list(PATHS))


@paths
@pytest.mark.parametrize("gate", [TIGHT, TIGHT_HALVES, mx.Gate("gelu"), mx.Gate("gelu_tanh", limit=0.75)])
def test_nan_scales_poison_both_gradients(path, gate):
    """NaN in either projection of an output makes its h, dg and du NaN, also
    where the other projection is past a clamp; nothing else changes."""
    need_gpu()
    ea, eb, M, N = PATHS[path]
    rng = np.random.default_rng(6)
    qa, _ = operand(rng, M, 160, ea)
    qb, _ = operand(rng, 2 * N, 160, eb, std=0.12)
    gate_row, up_row = (lambda c: c, lambda c: N + c) if gate.layout == "halves" else \
        (lambda c: 2 * c, lambda c: 2 * c + 1)
    dh = torch.ones(M, N, device="cuda")
    banner(f"NaN scales, {path}, {gate}")
    run = lambda: (host(mx.gemm_gated(qa, qb, gate, F32)), host(mx.gemm_gated_backward(qa, qb, dh, gate, F32)))
    h0, dP0 = run()
    assert np.isfinite(h0).all() and np.isfinite(dP0).all()
    qa.scales[2, 3] = 0xFF
    qb.scales[gate_row(4), 0] = 0xFF
    qb.scales[up_row(N - 1), 4] = 0xFF
    h, dP = run()
    want = np.zeros((M, N), bool)
    want[2], want[:, 4], want[:, N - 1] = True, True, True
    assert np.array_equal(np.isnan(h), want) and np.array_equal(h[~want], h0[~want])
    split = (lambda P: (P[:, :N], P[:, N:])) if gate.layout == "halves" else (lambda P: (P[:, 0::2], P[:, 1::2]))
    for part, d, d0 in zip(("dg", "du"), split(dP), split(dP0)):
        assert np.array_equal(np.isnan(d), want), part
        assert np.array_equal(d[~want], d0[~want]), part


def even(n):
    return n + (n & 1)


def aligned_case(M, N, K, gate, ea, eb, seed=0):
    """bf16 H, dH and dP at even strides and 4-byte aligned first columns, where
    the pipelines read and write whole lines; a tile's worth of rows behind the
    outputs, and columns around them, must stay as they were."""
    rng = np.random.default_rng([seed, M, N, K])
    qa, a = operand(rng, M, K, ea)
    qb, b = operand(rng, 2 * N, K, eb, std=1.5 / np.sqrt(K))
    P, e = projections(a, b, ea == eb == "e2m1")
    buf = torch.full((M + 260, even(N + 4)), 3.0, dtype=BF, device="cuda")
    mx.gemm_gated(qa, qb, gate, out=buf[1:M + 1, 2:N + 2])
    got = host(buf.float())
    ref, tol = forward_ref(P, e, gate)
    check(got[1:M + 1, 2:N + 2], ref, tol, True, what="h")
    got[1:M + 1, 2:N + 2] = 3.0
    assert np.all(got == 3.0), "written outside h"
    dh = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32)).to(BF)
    dhd = torch.full((M + 1, even(N + 4)), float("nan"), dtype=BF, device="cuda")
    dhd[:M, 2:N + 2] = dh.cuda()
    buf = torch.full((M + 260, 2 * N + 6), 3.0, dtype=BF, device="cuda")
    mx.gemm_gated_backward(qa, qb, dhd[:M, 2:N + 2], gate, out=buf[1:M + 1, 2:2 * N + 2])
    got = host(buf.float())
    ref, tol, alt = backward_ref(P, e, dh.double().numpy(), gate)
    check(got[1:M + 1, 2:2 * N + 2], ref, tol, True, alt, "dP")
    got[1:M + 1, 2:2 * N + 2] = 3.0
    assert np.all(got == 3.0), "written outside dP"


@pytest.mark.parametrize("ea,eb,M,N,K", [
    ("e2m1", "e2m1", 1100, 1900, 288), ("e2m1", "e2m1", 1025, 1857, 96), ("e2m1", "e2m1", 1279, 1794, 544),
    ("e4m3", "e4m3", 1100, 3700, 160), ("e4m3", "e5m2", 1025, 3713, 96), ("e2m3", "e3m2", 1279, 3586, 96),
    ("e2m1", "e2m1", 420, 900, 160), ("e4m3", "e2m1", 129, 1900, 160), ("e2m1", "e2m1", 33, 48, 160)])
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_whole_lines_of_bf16(ea, eb, M, N, K, layout):
    """Row tiles of 1 to 255 rows, column tiles that end at even and odd columns,
    both orders of the gate and up columns."""
    need_gpu()
    banner(f"gated bf16 lines {ea}/{eb} {M}x{N}x{K} {layout}")
    aligned_case(M, N, K, mx.Gate("silu", 1.702, 1.25, 1.0, layout), ea, eb)


@pytest.mark.parametrize("counts,N", [([1] * 39 + [33], 720), ([700, 0, 3, 256, 257, 1, 0], 720),
                                      ([1025, 1, 0, 511, 1], 641)])
@pytest.mark.parametrize("ea,eb", [("e2m1", "e2m1"), ("e4m3", "e4m3"), ("e4m3", "e2m1")])
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_grouped_bf16(counts, N, ea, eb, layout):
    """bf16 H, dH and dP (the default type) of one-row, ragged and whole tiles:
    a row tile that wrote past its expert's rows would change the next one's."""
    need_gpu()
    K = 96
    rng = np.random.default_rng([19, len(counts), N])
    gate, E, total = mx.Gate("silu", 1.702, 1.25, 1.0, layout), len(counts), int(np.sum(counts))
    cap = total + 260
    off, qa, a, qb, bs = _grouped(rng, counts, cap, E, N, K, eb, ea, "2d" if N % 16 == 0 else "1d")
    banner(f"grouped gated bf16 {counts} {N} {ea}/{eb} {layout}")
    offd = to_dev(off)
    H = torch.full((cap, even(N)), 3.0, dtype=BF, device="cuda")
    mx.grouped_gemm_gated(qa, offd, qb, gate, out=H[:, :N])
    dh = torch.from_numpy(rng.standard_normal((cap, even(N))).astype(np.float32)).to(BF)
    dP = torch.full((cap, 2 * N + 2), 3.0, dtype=BF, device="cuda")
    mx.grouped_gemm_gated_backward(qa, offd, qb, dh.cuda()[:, :N], gate, out=dP[:, :2 * N])
    H, dP, dh = host(H.float()), host(dP.float()), dh.double().numpy()[:, :N]
    assert np.all(H[total:] == 3.0) and np.all(dP[total:] == 3.0)
    assert np.all(H[:, N:] == 3.0) and np.all(dP[:, 2 * N:] == 3.0)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        P, err = projections(a[lo:hi], bs[e], ea == eb == "e2m1")
        ref, tol = forward_ref(P, err, gate)
        check(H[lo:hi, :N], ref, tol, True, what=f"h of expert {e}")
        ref, tol, alt = backward_ref(P, err, dh[lo:hi], gate)
        check(dP[lo:hi, :2 * N], ref, tol, True, alt, f"dP of expert {e}")


@paths
def test_graph_replays(path):
    """A captured forward and backward pass, replayed on changing inputs between
    eager calls."""
    need_gpu()
    ea, eb, M, N = PATHS[path]
    rng = np.random.default_rng(31)
    qb, _ = operand(rng, 2 * N, 288, eb, std=0.1)
    inputs = [operand(rng, M, 288, ea)[0] for _ in range(3)]
    qa = operand(rng, M, 288, ea)[0]
    dh = torch.randn(M, N, device="cuda").to(BF)
    run = lambda q: (mx.gemm_gated(q, qb, CLAMPED), mx.gemm_gated_backward(q, qb, dh, CLAMPED))
    banner(f"gated graph, {path}")
    run(qa)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(qa)
    for q in inputs:
        qa.codes.copy_(q.codes)
        qa.scales.copy_(q.scales)
        dh.normal_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, run(q)))


@pytest.mark.parametrize("elem", ["e2m1", "e4m3"])
def test_grouped_graph_replays_with_other_offsets(elem):
    """The offsets are read on the device: a replay follows them."""
    need_gpu()
    E, N, K, cap = 6, 720, 288, 1300
    rng = np.random.default_rng(33)
    _, qa, _, qb, _ = _grouped(rng, [cap], cap, E, N, K, elem, elem)
    offd = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    dh = torch.randn(cap, N, device="cuda").to(BF)
    H, dP = torch.empty(cap, N, dtype=BF, device="cuda"), torch.empty(cap, 2 * N, dtype=BF, device="cuda")
    run = lambda h, p: (mx.grouped_gemm_gated(qa, offd, qb, CLAMPED, out=h),
                        mx.grouped_gemm_gated_backward(qa, offd, qb, dh, CLAMPED, out=p))
    banner(f"grouped gated graph {elem}")
    run(H, dP)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(H, dP)
    for counts in ([300, 0, 1, 500, 255, 3], [0, 0, 0, 0, 0, 1300], [1, 1, 1, 1, 1, 1], [256, 257, 0, 0, 700, 0]):
        offd.copy_(torch.tensor(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)))
        H.fill_(3.0)
        dP.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        h, p = torch.full_like(H, 3.0), torch.full_like(dP, 3.0)
        run(h, p)
        assert torch.equal(h, H) and torch.equal(p, dP), counts


@paths
def test_k_of_zero(path):
    """Projections of nothing are zero: h = act(0) ..., dg = act'(0) up_shift."""
    need_gpu()
    ea, eb, M, N = PATHS[path]
    e = lambda r, elem: mx.MXTensor(torch.full((r, 16), 0x77, dtype=torch.uint8, device="cuda"),
                                    torch.full((r, 16), 0xFF, dtype=torch.uint8, device="cuda"), r, 0, "1d", elem)
    banner(f"gated K = 0, {path}")
    gate = mx.Gate(up_shift=2.0)
    assert np.all(host(mx.gemm_gated(e(M, ea), e(2 * N, eb), gate, F32)) == 0.0)
    dP = host(mx.gemm_gated_backward(e(M, ea), e(2 * N, eb), torch.ones(M, N, device="cuda"), gate, F32))
    assert np.all(dP[:, 0::2] == 1.0) and np.all(dP[:, 1::2] == 0.0)


@paths
def test_backward_same_bits(path):
    """The same bits on every run and on another stream."""
    need_gpu()
    ea, eb, M, N = PATHS[path]
    rng = np.random.default_rng(8)
    qa, qb = operand(rng, M, 2912, ea)[0], operand(rng, 2 * N, 2912, eb, std=0.1)[0]
    dh = torch.randn(M, N, device="cuda")
    banner(f"gated backward repeated, {path}")
    first = mx.gemm_gated_backward(qa, qb, dh, CLAMPED, F32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(s):
            again = mx.gemm_gated_backward(qa, qb, dh, CLAMPED, F32)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(first, again)
