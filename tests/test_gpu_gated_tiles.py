"""The gated block's tile kernels at sizes past the ranges of the kernel for few
rows (more than 768 of its 32 x 16 tiles, grouped more than 1536 and 8 rows per
expert): 128 x 64 tiles up to 256 workgroups (512 with elements wider than
MXFP4), the 256-row pipelines above.  Formulas and tolerances are those of
test_gpu_gated."""
import numpy as np
import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx
from gpu_util import banner, host, need_gpu, to_dev
from test_gpu_gated import (CLAMPED, ELEMS, TIGHT, _grouped, backward_ref, check, forward_ref, operand, projections,
                            run_case)

pytestmark = pytest.mark.gpu

GATES = [mx.Gate(), mx.Gate("gelu", layout="halves"), mx.Gate("gelu_tanh", limit=2.0), CLAMPED,
         mx.Gate("gelu", limit=0.75, up_shift=-0.5)]


@pytest.mark.parametrize("ea", ELEMS)
@pytest.mark.parametrize("eb", ELEMS)
def test_tile_element_types(ea, eb):
    """Every pair of element types, K ending one block into a stage."""
    need_gpu()
    run_case(420, 900, 288, mx.Gate("silu", 1.702, 1.25, 1.0, "halves"), ea, eb, out=torch.bfloat16,
             dh_dtype=torch.bfloat16)


@pytest.mark.parametrize("ea,eb", [("e2m1", "e2m1"), ("e4m3", "e5m2"), ("e2m3", "e3m2"), ("e3m2", "e2m1")])
@pytest.mark.parametrize("M,N,K", [(400, 960, 32), (513, 833, 96), (897, 449, 128), (417, 897, 480), (512, 800, 544),
                                   (420, 890, 2912)])
def test_tile_depths(ea, eb, M, N, K):
    """One stage, fewer stages than the ring has slots, whole and partial last
    stages; rows and columns that end 1 into a tile and at its end."""
    need_gpu()
    run_case(M, N, K, TIGHT, ea, eb)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("ea,M,N", [("e2m1", 420, 900), ("e4m3", 420, 900), ("e2m1", 1100, 1900), ("e4m3", 1100, 3700)])
def test_tile_and_pipeline_activations(gate, ea, M, N):
    need_gpu()
    run_case(M, N, 160, gate, ea, ea, out=torch.bfloat16, dh_dtype=torch.float32)


@pytest.mark.parametrize("a_block,b_block,layout", [("1d", "2d", "interleaved"), ("1d", "2d", "halves"),
                                                    ("2d", "1d", "halves"), ("2d", "2d", "interleaved")])
@pytest.mark.parametrize("elem,M,N", [("e2m1", 448, 912), ("e4m3", 448, 912), ("e2m1", 1120, 1904),
                                      ("e4m3", 1120, 3696)])
def test_tile_and_pipeline_two_dimensional_scales(elem, M, N, a_block, b_block, layout):
    need_gpu()
    run_case(M, N, 160, mx.Gate("silu", 1.702, 1.25, 1.0, layout), elem, elem, a_block=a_block, b_block=b_block)


@pytest.mark.parametrize("pad", [1, 2, 4])
@pytest.mark.parametrize("ea,eb", [("e2m1", "e2m1"), ("e4m3", "e4m3"), ("e4m3", "e2m3")])
@pytest.mark.parametrize("M,N,K", [(420, 900, 608), (1100, 1900, 288)])
def test_tile_scale_row_strides(pad, ea, eb, M, N, K):
    """Scale rows that start at any byte, or 4-byte ones."""
    need_gpu()
    run_case(M, N, K, CLAMPED, ea, eb, pad=pad)


@pytest.mark.parametrize("ea,eb,M,N,K,layout", [
    ("e2m1", "e2m1", 1100, 1900, 96, "halves"), ("e2m1", "e2m1", 1537, 1301, 256, "interleaved"),
    ("e2m1", "e2m1", 1025, 1857, 544, "halves"), ("e2m1", "e2m1", 1025, 1857, 800, "interleaved"),
    ("e4m3", "e5m2", 1100, 3700, 96, "interleaved"), ("e4m3", "e4m3", 1537, 2600, 256, "halves"),
    ("e2m3", "e4m3", 1025, 3713, 288, "interleaved"), ("e3m2", "e3m2", 1025, 3713, 544, "halves"),
    ("e2m1", "e4m3", 1025, 3713, 288, "halves")])
def test_pipelines(ea, eb, M, N, K, layout):
    """Ragged rows and columns and K tails of the 256-row pipelines (a mixed
    MXFP4 pair keeps to 128 x 64 tiles)."""
    need_gpu()
    run_case(M, N, K, mx.Gate("silu", 1.702, 1.25, 1.0, layout), ea, eb, out=torch.bfloat16, dh_dtype=torch.bfloat16)


@pytest.mark.parametrize("ea,eb", [("e2m1", "e2m1"), ("e4m3", "e5m2"), ("e2m3", "e3m2"), ("e3m2", "e2m1")])
@pytest.mark.parametrize("M,N,K", [(97, 2880, 96), (33, 6000, 32), (128, 2890, 544), (100, 2881, 2880)])
def test_few_rows_of_many_columns(ea, eb, M, N, K):
    """More than 2.5 workgroups per CU of the kernel for few rows: K split over
    2 waves, with none, one or several pieces each."""
    need_gpu()
    run_case(M, N, K, TIGHT, ea, eb)


@pytest.mark.parametrize("counts,N,K", [([1] * 39 + [33], 720, 288), ([700, 0, 3, 256, 257, 0], 720, 288), ([1025, 1, 0, 511], 640, 96)])
@pytest.mark.parametrize("ea,eb", [("e2m1", "e2m1"), ("e4m3", "e4m3"), ("e2m3", "e5m2"), ("e4m3", "e2m1")])
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_grouped_tiles(counts, N, K, ea, eb, layout):
    """Experts without rows, with one row, with whole and ragged 256-row tiles."""
    need_gpu()
    rng = np.random.default_rng([17, len(counts), N, K])
    gate, E, total = mx.Gate("silu", 1.702, 1.25, 1.0, layout), len(counts), int(np.sum(counts))
    cap = total + 5
    off, qa, a, qb, bs = _grouped(rng, counts, cap, E, N, K, eb, ea)
    banner(f"grouped gated tiles {counts} {N}x{K} {ea}/{eb} {layout}")
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


@pytest.mark.parametrize("elem,M,N", [("e2m1", 420, 900), ("e4m3", 420, 900), ("e2m3", 420, 900), ("e2m1", 1100, 1900),
                                      ("e4m3", 1100, 3700), ("e2m3", 1100, 3700)])
def test_tile_and_pipeline_nan_scales(elem, M, N):
    """A NaN scale of an A row makes that row NaN, one of a gate or up row its
    column; codes and scales past K have no say in any output."""
    need_gpu()
    rng = np.random.default_rng(6)
    qa, a = operand(rng, M, 160, elem)
    qb, b = operand(rng, 2 * N, 160, elem, std=0.1)
    qa.scales[2, 3] = 0xFF
    qb.scales[2 * 4, 0] = 0xFF                       # gate of column 4
    qb.scales[2 * (N - 1) + 1, 4] = 0xFF             # up of the last column
    banner(f"gated tiles NaN scales {M}x{N} {elem}")
    h = host(mx.gemm_gated(qa, qb, TIGHT, torch.float32))
    want = np.zeros((M, N), bool)
    want[2], want[:, 4], want[:, N - 1] = True, True, True
    assert np.array_equal(np.isnan(h), want)


@pytest.mark.parametrize("elem,M,N", [("e2m1", 420, 900), ("e4m3", 420, 900), ("e2m1", 1100, 1900),
                                      ("e4m3", 1100, 3700)])
def test_tile_and_pipeline_same_bits(elem, M, N):
    """The same bits on every run and on another stream."""
    need_gpu()
    rng = np.random.default_rng(8)
    qa, qb = operand(rng, M, 2912, elem)[0], operand(rng, 2 * N, 2912, elem, std=0.1)[0]
    banner(f"gated tiles repeated {M}x{N} {elem}")
    first = mx.gemm_gated(qa, qb, CLAMPED, torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(s):
            again = mx.gemm_gated(qa, qb, CLAMPED, torch.float32)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(first, again)
