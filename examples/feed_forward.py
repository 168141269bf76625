"""The feed-forward half of a transformer block, trained and served in MXFP4.

    y = x + dropout( W2 . gated( W1 . norm(x) ) )

Training step: layer norm, the activations quantized along K, the gated block
(both projections, the activation and the product in one kernel) on W1 in
32 x 32 tiles, its output quantized, the down projection, dropout added to the
residual; then every gradient.  The backward products follow the library's
MXFP4 recipe: gradients quantized with stochastic rounding, the data gradients
through the exact transposes of the forward weights, the weight gradients from
both operands quantized along the token dimension with the randomized Hadamard
transform.  Kept for the backward pass are x, the normalized rows (bf16, for the
weight gradient, and quantized), the block's output, the norm's statistics and
the quantized weights: the gated block recomputes its projections and the
dropout mask comes from its seed.

    python examples/feed_forward.py            # train on a fixed batch, then serve one token
"""
import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_microscaling_quantization_mx_amd as mx  # noqa: E402

MASK = 0x1234ABCD            # signs of the Hadamard transform of the weight gradients


@dataclass
class FeedForward:
    """Weights (float32 masters) and settings of one block."""
    w1: torch.Tensor         # [2 hidden, width], gate and up rows interleaved
    w2: torch.Tensor         # [width, hidden]
    norm_w: torch.Tensor     # [width]
    norm_b: torch.Tensor     # [width]
    gate: mx.Gate = mx.Gate("silu", alpha=1.702, limit=7.0, up_shift=1.0)
    p: float = 0.1

    @classmethod
    def random(cls, width, hidden, seed=0, **kw):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda r, c: torch.randn(r, c, device="cuda", generator=g) * c ** -0.5
        return cls(rand(2 * hidden, width), rand(width, hidden), torch.ones(width, device="cuda"),
                   torch.zeros(width, device="cuda"), **kw)

    def quantized(self):
        """Both weights in 32 x 32 tiles, the forward operands."""
        return mx.quantize(self.w1, block="2d"), mx.quantize(self.w2, block="2d")

    def forward(self, x, step, training=True, weights=None):
        """y for x [tokens, width] bf16, and what the backward pass needs."""
        q1, q2 = weights or self.quantized()
        n, mean, rstd = mx.layer_norm(x, self.norm_w, self.norm_b)
        qn = mx.quantize(n)
        h = mx.gemm_gated(qn, q1, self.gate)
        d = mx.gemm(mx.quantize(h), q2, torch.bfloat16)
        y = mx.dropout(d, self.p if training else 0.0, seed=step, offset=1, residual=x)
        return y, (x, mean, rstd, n, qn, h, q1, q2, step)

    def backward(self, dy, saved):
        """Gradients of x and of every weight for dy [tokens, width] bf16."""
        x, mean, rstd, n, qn, h, q1, q2, step = saved
        sr = dict(rounding="sr", seed=step)
        wide = dict(axis="dim0", rht_mask=MASK, **sr)       # along the tokens, for the weight gradients
        dd = mx.dropout(dy, self.p, seed=step, offset=1)
        dh = mx.gemm(mx.quantize(dd, offset=2, **sr), mx.transpose(q2), torch.bfloat16)
        dw2 = mx.gemm(mx.quantize(dd, offset=3, **wide), mx.quantize(h, offset=4, **wide))
        dp = mx.gemm_gated_backward(qn, q1, dh, self.gate)
        dn = mx.gemm(mx.quantize(dp, offset=5, **sr), mx.transpose(q1), torch.bfloat16)
        dw1 = mx.gemm(mx.quantize(dp, offset=6, **wide), mx.quantize(n, offset=7, **wide))
        dx, dnw, dnb = mx.layer_norm_backward(dn, x, mean, rstd, self.norm_w)
        return dx + dy, dict(w1=dw1, w2=dw2, norm_w=dnw, norm_b=dnb)


def train(block, x, target, steps, lr):
    """Gradient descent on the mean squared error, each weight moved by `lr` of
    its size (of 1 for the norm's) along its gradient; the loss of every step."""
    losses = []
    for step in range(steps):
        y, saved = block.forward(x, step)
        diff = y.float() - target.float()
        losses.append(float(diff.square().mean()))
        dy = (diff * (2 / diff.numel())).to(torch.bfloat16)
        _, grads = block.backward(dy, saved)
        for name, g in grads.items():
            w = getattr(block, name)
            size = w.norm() if w.dim() == 2 else w.numel() ** 0.5
            w.sub_(g * (lr * size / g.norm()))
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=2880)
    ap.add_argument("--hidden", type=int, default=2880)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.05)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.width, device="cuda", generator=g).to(torch.bfloat16)
    # the target: x plus what another block of the same shape adds to it
    target, _ = FeedForward.random(a.width, a.hidden, seed=2).forward(x, 0, training=False)
    block = FeedForward.random(a.width, a.hidden, seed=3)
    losses = train(block, x, target, a.steps, a.lr)
    print("loss", " ".join(f"{v:.4f}" for v in losses))
    # serving: the weights quantized once, one token at a time
    weights = block.quantized()
    y, _ = block.forward(x[:1], 0, training=False, weights=weights)
    full, _ = block.forward(x, 0, training=False, weights=weights)
    print("one token against the batch: largest difference %.4f of %.4f" %
          (float((y - full[:1]).abs().max()), float(full[:1].abs().max())))


if __name__ == "__main__":
    main()
