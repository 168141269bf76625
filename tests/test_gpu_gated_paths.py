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
    "few, 2 waves": ("e4m3", "e2m1", 100, 2881),
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
