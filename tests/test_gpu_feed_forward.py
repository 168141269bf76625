"""The feed-forward block of examples/feed_forward.py: norm, gated block, down
projection and dropout together, forward and backward, against the block in
float64 without quantization, and its training and serving paths."""
import os
import sys

import numpy as np
import pytest
import torch

from gpu_util import banner, need_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def reference(block, x, step, keep):
    """The block in float64 autograd: y and a function of dy to the gradients.
    keep: the dropout factors (0 or 1 / (1 - p)) as drawn on the GPU."""
    leaves = [t.double().requires_grad_() for t in (x, block.w1, block.w2, block.norm_w, block.norm_b)]
    x, w1, w2, nw, nb = leaves
    n = torch.nn.functional.layer_norm(x, x.shape[1:], nw, nb)
    P = n @ w1.t()
    g, u, lim = P[:, 0::2].clamp(max=7.0), P[:, 1::2].clamp(-7.0, 7.0), 7.0
    y = x + keep * (((u + 1) * g * torch.sigmoid(1.702 * g)) @ w2.t())
    return y, lambda dy: torch.autograd.grad(y, leaves, dy.double())


def rel(a, b):
    return float(((a.double() - b).norm() / b.norm()).detach())


@pytest.mark.parametrize("tokens,width,hidden", [(512, 640, 768), (96, 320, 288)])
def test_forward_and_gradients_follow_the_block(tokens, width, hidden):
    """MXFP4 operands cost 10-20 % per product (the linear layer's tests); the
    block's output and gradients stay within what three products in a row of
    that error allow, and point the same way."""
    need_gpu()
    import feed_forward as ff
    import mxfp4_microscaling_quantization_mx_amd as mx
    block = ff.FeedForward.random(width, hidden, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(tokens, width, device="cuda", generator=g).to(torch.bfloat16)
    dy = torch.randn(tokens, width, device="cuda", generator=g).to(torch.bfloat16)
    banner(f"feed forward {tokens}x{width}x{hidden}")
    y, saved = block.forward(x, step=9)
    dx, grads = block.backward(dy, saved)
    keep = mx.dropout(torch.ones(tokens, width, device="cuda"), block.p, seed=9, offset=1).double()
    ry, back = reference(block, x, 9, keep)
    rdx, rw1, rw2, rnw, rnb = back(dy)
    errs = dict(y=rel(y - x, ry - x.double()), dx=rel(dx.float() - dy.float(), rdx - dy.double()),
                w1=rel(grads["w1"], rw1), w2=rel(grads["w2"], rw2), norm_w=rel(grads["norm_w"], rnw),
                norm_b=rel(grads["norm_b"], rnb))
    print("[feed forward] relative errors", {k: round(v, 3) for k, v in errs.items()})
    # an error of 0.6 of the norm still leaves a cosine of 0.8 with the exact gradient
    assert all(v < 0.6 for v in errs.values()), errs


def test_training_lowers_the_loss_and_serving_agrees():
    need_gpu()
    import feed_forward as ff
    banner("feed forward training")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(512, 640, device="cuda", generator=g).to(torch.bfloat16)
    target, _ = ff.FeedForward.random(640, 512, seed=2, p=0.0).forward(x, 0)
    block = ff.FeedForward.random(640, 512, seed=3, p=0.05)
    losses = ff.train(block, x, target, steps=20, lr=0.05)
    print("[feed forward] losses", np.round(losses, 4))
    assert all(np.isfinite(losses)) and losses[-1] < 0.7 * losses[0]
    # one token's products take other kernels than a batch's: the same sums in
    # another order, so a few codes of the quantized h may differ
    weights = block.quantized()
    full, _ = block.forward(x, 0, training=False, weights=weights)
    one, _ = block.forward(x[:1], 0, training=False, weights=weights)
    assert rel(one, full[:1].double()) < 0.05
