"""examples/experts.py: a training step moves every weight by `lr` of its size against
the gradient that the backward pass gives for that batch and step."""
import copy
import os
import sys

import pytest
import torch

from gpu_util import banner, need_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
NAMES = ("wr", "w1", "b1", "w2", "b2")


def test_steps_go_against_the_gradient():
    need_gpu()
    import experts as ex
    banner("experts training steps")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(200, 320, device="cuda", generator=g).to(torch.bfloat16)
    target, _ = ex.Experts.random(8, 320, 256, seed=2, top=2).forward(x)
    block = ex.Experts.random(8, 320, 256, seed=3, top=2)
    own, lr = copy.deepcopy(block), 0.02
    losses = ex.train(block, x, target, steps=2, lr=lr)
    for step in range(2):
        y, saved = own.forward(x)
        diff = y.double() - target.double()
        assert abs(losses[step] - float(diff.square().mean())) <= 1e-5 * losses[step]
        _, grads = own.backward((diff.float() * (2 / diff.numel())).to(torch.bfloat16), saved, step)
        for name in NAMES:
            w, d = getattr(own, name), grads[name].double()
            assert float(d.norm()) > 0
            setattr(own, name, (w.double() - d * (lr * w.double().norm() / d.norm())).float())
    for name in NAMES:
        w, want = getattr(block, name), getattr(own, name)
        # float32 norms of n values, one product and one difference of float32 numbers per step
        assert float((w - want).abs().max()) <= 2 * 2.0 ** -20 * float(want.abs().max()), name
