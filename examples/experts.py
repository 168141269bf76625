"""The expert half of a transformer block, trained and served in MXFP4.

    y[t] = x[t] + sum_j w[t, j] ( W2_e gelu( W1_e x[t] + b1_e ) + b2_e ),   e = ids[t, j]

Forward: the router's logits (a float32 product), the top experts of every token and
their weights, the slots sorted by expert, each token quantized once into its sorted
rows, two linear layers per expert with bias and activation in their epilogues, and
the weighted sum back on the residual stream.  The backward pass goes the same way:
gradients quantized with stochastic rounding, the data gradients through the exact
transposes of the forward weights, the weight gradients from both operands quantized
along the tokens with the randomized Hadamard transform.  Kept for it are x, the
routing, the sorted quantized rows, h and the experts' outputs; the first layer's
pre-activation is recomputed.

    python examples/experts.py            # train on a fixed batch, then serve one token
"""
import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_microscaling_quantization_mx_amd as mx  # noqa: E402

MASK = 0x1234ABCD            # signs of the Hadamard transform of the weight gradients
ACT = "gelu_tanh"


@dataclass
class Experts:
    """Weights (float32 masters) and settings of one block."""
    wr: torch.Tensor         # [experts, width], the router
    w1: torch.Tensor         # [experts, hidden, width]
    b1: torch.Tensor         # [experts, hidden]
    w2: torch.Tensor         # [experts, width, hidden]
    b2: torch.Tensor         # [experts, width]
    top: int = 4
    router: mx.Router = mx.Router()

    @classmethod
    def random(cls, experts, width, hidden, seed=0, **kw):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g) * s[-1] ** -0.5
        return cls(rand(experts, width), rand(experts, hidden, width), rand(experts, hidden), rand(experts, width, hidden),
                   rand(experts, width), **kw)

    def quantized(self):
        """Both weights of every expert in 32 x 32 tiles, the forward operands."""
        return tuple(stacked(lambda e, out, w=w: mx.quantize(w[e], block="2d", out=out), w.shape) for w in (self.w1, self.w2))

    def forward(self, x, weights=None):
        """y for x [tokens, width] bf16, and what the backward pass needs."""
        q1, q2 = weights or self.quantized()
        logits = x.float() @ self.wr.t()
        ids, w = mx.route(logits, self.top, self.router)
        offsets, _, dest = mx.expert_sort(ids, self.wr.shape[0])
        qx = mx.quantize_scatter(x, dest, self.top)
        h = mx.grouped_linear(qx, offsets, q1, bias=self.b1, act=ACT)
        y = mx.grouped_linear(mx.quantize(h), offsets, q2, bias=self.b2)
        out = mx.expert_combine(y, dest, w, residual=x)
        return out, (x, logits, ids, w, offsets, dest, qx, h, y, q1, q2)

    def backward(self, dout, saved, step):
        """Gradients of x and of every weight for dout [tokens, width] bf16."""
        x, logits, ids, w, offsets, dest, qx, h, y, q1, q2 = saved
        sr = dict(rounding="sr", seed=step)
        dy, dw = mx.expert_combine_backward(dout, y, dest, w)
        dh = mx.grouped_gemm(mx.quantize(dy, offset=1, **sr), offsets, transposed(q2))
        dp = mx.grouped_linear_backward(qx, offsets, q1, dh, bias=self.b1, act=ACT)
        dxs = mx.grouped_gemm(mx.quantize(dp, offset=2, **sr), offsets, transposed(q1))
        dlogits = mx.route_backward(dw, logits, ids, self.router)
        dx = mx.expert_combine(dxs, dest, residual=dout)
        dx = (dx.float() + dlogits @ self.wr).to(x.dtype)
        xs = mx.expert_dispatch(x, dest)
        return dx, dict(wr=dlogits.t() @ x.float(), w1=weight_grad(dp, xs, offsets, step, 3), b1=mx.bias_grad(dp, offsets),
                        w2=weight_grad(dy, h, offsets, step, 5), b2=mx.bias_grad(dy, offsets))


def stacked(make, shape):
    """An operand of experts [E, rows, K] with 2-D blocks, filled by make(e, out)."""
    q = mx.empty_mx(shape[1], shape[2], "2d", experts=shape[0])
    for e in range(shape[0]):
        make(e, mx.expert(q, e))
    return q


def transposed(q):
    return stacked(lambda e, out: mx.transpose(mx.expert(q, e), out=out), (q.codes.shape[0], q.K, q.rows))


def weight_grad(dp, x, offsets, step, offset):
    """dW_e = dp_e^T x_e for the rows of every expert, quantized along them (padded
    with zero rows to whole blocks of 32)."""
    out = torch.zeros(offsets.numel() - 1, dp.shape[1], x.shape[1], device=dp.device)
    ends = offsets.tolist()
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi > lo:
            pad = lambda t: torch.nn.functional.pad(t[lo:hi], (0, 0, 0, -(hi - lo) % 32))
            q = lambda t, k: mx.quantize(pad(t), axis="dim0", rht_mask=MASK, rounding="sr", seed=step, offset=offset + k)
            mx.gemm(q(dp, 0), q(x, 1), out=out[e])
    return out


def train(block, x, target, steps, lr):
    """Gradient descent on the mean squared error, each weight moved by `lr` of its
    size along its gradient; the loss of every step."""
    losses = []
    for step in range(steps):
        y, saved = block.forward(x)
        diff = y.float() - target.float()
        losses.append(float(diff.square().mean()))
        _, grads = block.backward((diff * (2 / diff.numel())).to(torch.bfloat16), saved, step)
        for name, g in grads.items():
            w = getattr(block, name)
            w.sub_(g * (lr * w.norm() / g.norm().clamp_min(1e-20)))
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--width", type=int, default=2880)
    ap.add_argument("--hidden", type=int, default=2880)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--lr", type=float, default=0.05)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.width, device="cuda", generator=g).to(torch.bfloat16)
    # the target: x plus what another block of the same shape adds to it
    target, _ = Experts.random(a.experts, a.width, a.hidden, seed=2).forward(x)
    block = Experts.random(a.experts, a.width, a.hidden, seed=3)
    losses = train(block, x, target, a.steps, a.lr)
    print("loss", " ".join(f"{v:.4f}" for v in losses))
    # serving: the weights quantized once, one token at a time
    weights = block.quantized()
    y, _ = block.forward(x[:1], weights)
    full, _ = block.forward(x, weights)
    print("one token against the batch: largest difference %.4f of %.4f" %
          (float((y - full[:1]).abs().max()), float(full[:1].abs().max())))


if __name__ == "__main__":
    main()
