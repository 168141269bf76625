"""examples/experts.py step by step: its output and every gradient against the same
chain in float64 on the dequantized operands.

Each step of the chain takes the step before it rounded to bf16, as the block does,
and quantizes it with the same draws, so what is left between the two is float32
accumulation, now and then a bf16 rounding that falls the other way, and the codes
that such a rounding moves: bf16's 2^-9 of a value at most, far below the 10-20 % that
the quantization itself costs.  A wrong row, expert, transpose, seed or weight would
be an error of the size of the result."""
import os
import sys

import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx
from gpu_util import banner, need_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def deq(q):
    return mx.dequantize(q).double()


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("tokens,experts,width,hidden,top,score", [(512, 8, 320, 416, 2, "softmax"), (96, 16, 288, 256, 4, "sigmoid"),
                                                                   (3, 32, 64, 96, 4, "softmax")])
def test_output_and_gradients_are_the_chain(tokens, experts, width, hidden, top, score):
    need_gpu()
    import experts as ex
    block = ex.Experts.random(experts, width, hidden, seed=5, top=top, router=mx.Router(score, True, 1.0))
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(tokens, width, device="cuda", generator=g).to(BF)
    dout = torch.randn(tokens, width, device="cuda", generator=g).to(BF)
    step = 9
    banner(f"experts chain {tokens} tokens {experts}x{width}x{hidden} top {top} {score}")
    out, saved = block.forward(x)
    dx, grads = block.backward(dout, saved, step)

    q1, q2 = block.quantized()
    leaf = (x.float() @ block.wr.t()).double().requires_grad_()
    ids = torch.sort(leaf.detach(), dim=1, descending=True, stable=True)[1][:, :top]
    s = leaf.gather(1, ids)
    w = torch.softmax(s, 1) if score == "softmax" else torch.sigmoid(s) / torch.sigmoid(s).sum(1, keepdim=True)
    order = torch.argsort(ids.reshape(-1), stable=True)               # sorted row -> slot
    tok, slot_e = order // top, ids.reshape(-1)[order]
    wd = w.detach().reshape(-1)[order]
    counts = torch.bincount(slot_e, minlength=experts).tolist()
    ends = [0]
    for c in counts:
        ends.append(ends[-1] + c)
    spans = [(e, lo, hi) for e, (lo, hi) in enumerate(zip(ends, ends[1:])) if hi > lo]
    per = lambda f, n: torch.cat([f(e, slice(lo, hi)) for e, lo, hi in spans]) if spans else torch.zeros(0, n)
    W1 = [deq(mx.expert(q1, e)) for e in range(experts)]
    W2 = [deq(mx.expert(q2, e)) for e in range(experts)]
    xs = x[tok]
    qx = deq(mx.quantize(xs))
    P = per(lambda e, r: qx[r] @ W1[e].t() + block.b1[e].double(), hidden).requires_grad_()
    act = torch.nn.functional.gelu(P, approximate="tanh")
    h = act.detach().to(BF)
    qh = deq(mx.quantize(h))
    y = per(lambda e, r: qh[r] @ W2[e].t() + block.b2[e].double(), width).to(BF)
    ref = x.double().index_add(0, tok, y.double() * wd[:, None])
    errs = dict(out=rel(out.double() - x.double(), ref - x.double()))

    sr = dict(rounding="sr", seed=step)
    dy = (dout.double()[tok] * wd[:, None]).to(BF)
    dslot = (dout.double()[tok] * y.double()).sum(1)
    dw = torch.zeros(tokens * top, dtype=torch.float64, device="cuda").index_copy(0, order, dslot).view(tokens, top)
    dlogits, = torch.autograd.grad((w * dw).sum(), leaf)
    errs["wr"] = rel(grads["wr"], dlogits.t() @ x.double())
    qdy = deq(mx.quantize(dy, offset=1, **sr))
    dh = per(lambda e, r: qdy[r] @ W2[e], hidden).to(BF)
    slope, = torch.autograd.grad(act.sum(), P)
    dp = (dh.double() * slope).to(BF)
    qdp = deq(mx.quantize(dp, offset=2, **sr))
    dxs = per(lambda e, r: qdp[r] @ W1[e], width).to(BF)
    rdx = (dlogits @ block.wr.double()).index_add(0, tok, dxs.double())
    errs["dx"] = rel(dx.double() - dout.double(), rdx)
    add = lambda t: torch.zeros(experts, t.shape[1], dtype=torch.float64, device="cuda").index_add(0, slot_e, t.double())
    errs["b1"], errs["b2"] = rel(grads["b1"], add(dp)), rel(grads["b2"], add(dy))
    for name, a, b, off in (("w1", dp, xs, 3), ("w2", dy, h, 5)):
        ref = torch.zeros_like(grads[name], dtype=torch.float64)
        for e, lo, hi in spans:
            pad = lambda t: torch.nn.functional.pad(t[lo:hi], (0, 0, 0, -(hi - lo) % 32))
            q = lambda t, k: deq(mx.quantize(pad(t), axis="dim0", rht_mask=ex.MASK, offset=off + k, **sr))
            ref[e] = q(a, 0) @ q(b, 1).t()
        errs[name] = rel(grads[name], ref)
    print("[experts chain] relative errors", {k: round(e, 5) for k, e in errs.items()})
    # out - x and dx - dout come from bf16 sums with x and dout: half an ulp of those, 2^-9
    # of values that are at most a few times the difference; the rest as above
    assert all(e < 0.02 for e in errs.values()), errs


def test_training_runs_and_one_token_is_served():
    need_gpu()
    import experts as ex
    banner("experts training")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(200, 320, device="cuda", generator=g).to(BF)
    target, _ = ex.Experts.random(8, 320, 256, seed=2, top=2).forward(x)
    block = ex.Experts.random(8, 320, 256, seed=3, top=2)
    losses = ex.train(block, x, target, steps=3, lr=0.02)
    assert len(losses) == 3 and all(v == v and v < float("inf") for v in losses)
    weights = block.quantized()
    full, _ = block.forward(x, weights)
    one, _ = block.forward(x[:1], weights)
    # one token's products take other kernels than a batch's: the same sums in another
    # order, so a few codes of the quantized h may differ
    assert rel(one, full[:1]) < 0.05
