"""Rows to their places sorted by expert and back, and bias gradients, on the GPU
against 64-bit forms."""
import numpy as np
import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx
from experts_util import TINY, U, f64, half_step, sort_slots, strided
from gpu_util import banner, host, need_gpu

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")
# columns: within a piece, at its borders, odd, a wave's worth and around it, several waves
WIDTHS = [1, 3, 4, 7, 8, 9, 64, 100, 255, 256, 257, 511, 513, 1111, 2880, 8195]


def routing(T, top, E, drop, seed):
    g = np.random.default_rng([seed, T, top, E])
    ids = np.stack([g.permutation(E)[:top] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, top), np.int32)
    ids[g.random(ids.shape) < drop] = -1
    offsets, _, dest = sort_slots(ids, E)
    w = torch.from_numpy(g.random((T, top)).astype(np.float32)).cuda()
    return int(offsets[-1]), torch.from_numpy(dest).cuda(), w


def combine_ref(y, dest, w, r):
    """Sum and sum of magnitudes."""
    T, top = dest.shape
    s, m = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for j in range(top):
        live = np.flatnonzero((dest[:, j] >= 0) & (dest[:, j] < y.shape[0]))
        v = y[dest[live, j]] * (1.0 if w is None else w[live, j, None])
        s[live] += v
        m[live] += np.abs(v)
    return (s, m) if r is None else (s + r, m + np.abs(r))


def close(got, ref, tol):
    got = f64(got)
    assert got.shape == ref.shape
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / tol))


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_combine_and_gradients(C, dtype):
    need_gpu()
    for T, top, E, drop in ((1, 1, 2, 0.0), (5, 4, 8, 0.0), (67, 3, 5, 0.3), (33, 9, 16, 0.1)):
        banner(f"combine C={C} {dtype} T={T} top={top}")
        M, dest, w = routing(T, top, E, drop, C)
        # padded rows that start at odd elements, and contiguous ones
        for ld, shift in ((C + 5, 3), (C, 0)):
            y = strided((M, C), ld, shift, dtype, 1)
            r = strided((T, C), ld + 1, shift, dtype, 2)
            d = host(dest)
            for weight, res in ((w, None), (w, r), (None, None), (None, r)):
                out = mx.expert_combine(y, dest, weight, residual=res)
                s, m = combine_ref(f64(y), d, None if weight is None else f64(weight), None if res is None else f64(res))
                # top + 1 roundings of partial sums, then the type's
                close(out, s, (top + 1.01) * U * m + np.abs(s) * half_step(dtype) * 1.01 + TINY)
            dout = strided((T, C), ld + 2, 1, dtype, 3)
            dy, dw = mx.expert_combine_backward(dout, y, dest, w)
            ref_dy, ref_dw, mag = np.full((M, C), np.nan), np.zeros((T, top)), np.zeros((T, top))
            for t in range(T):
                for j in range(top):
                    if d[t, j] >= 0:
                        ref_dy[d[t, j]] = f64(w)[t, j] * f64(dout[t])
                        ref_dw[t, j] = f64(dout[t]) @ f64(y[d[t, j]])
                        mag[t, j] = np.abs(f64(dout[t])) @ np.abs(f64(y[d[t, j]]))
            assert not np.isnan(ref_dy).any()
            close(dy, ref_dy, np.abs(ref_dy) * (half_step(dtype) + U) * 1.01 + TINY)
            # a lane adds up at most 32 products, then 6 steps over lanes and 8 over waves
            close(dw, ref_dw, 48 * U * mag + TINY)
            xs = mx.expert_dispatch(dout, dest, rows_out=M)
            tok = np.zeros(M, np.int64)
            for t in range(T):
                tok[d[t][d[t] >= 0]] = t
            assert torch.equal(xs, dout[torch.from_numpy(tok).cuda()])


def test_dropped_slots_touch_nothing():
    """Entries of dest outside the rows: nothing is read or written for them, and
    what is not a number beside them stays out."""
    need_gpu()
    banner("combine dropped slots")
    C = 100
    y = torch.randn(3, C, device="cuda")
    y[0] = NAN                                           # the row that no slot names
    dest = torch.tensor([[1, -1], [3, 2], [-5, 2**31 - 1], [-2**31, 100]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, NAN], [NAN, 2.0], [NAN, NAN], [1.0, 1.0]], device="cuda")
    out = mx.expert_combine(y, dest, w)
    assert torch.equal(out[0], 0.5 * y[1]) and torch.equal(out[1], 2.0 * y[2]) and not out[2:].any()
    r = torch.randn(4, C, device="cuda")
    assert torch.equal(mx.expert_combine(y, dest, w, residual=r)[2:], r[2:])
    dout = torch.randn(4, C, device="cuda")
    dy = torch.full((3, C), 7.0, device="cuda")
    _, dw = mx.expert_combine_backward(dout, y, dest, w, out=dy)
    assert torch.equal(dy[0], torch.full((C,), 7.0, device="cuda"))
    assert torch.equal(dy[1], 0.5 * dout[0]) and torch.equal(dy[2], 2.0 * dout[1])
    live = torch.tensor([[True, False], [False, True], [False, False], [False, False]], device="cuda")
    assert not dw[~live].any() and torch.isfinite(dw).all()
    xs = torch.full((3, C), 7.0, device="cuda")
    mx.expert_dispatch(dout, dest, out=xs)
    assert torch.equal(xs[0], dy[0]) and torch.equal(xs[1], dout[0]) and torch.equal(xs[2], dout[1])


def test_nan_and_inf_pass_through():
    need_gpu()
    banner("combine NaN and Inf")
    y = torch.tensor([[1.0, NAN, float("inf"), 0.0], [2.0, 1.0, 1.0, float("-inf")]], device="cuda")
    dest = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    out = mx.expert_combine(y, dest, torch.tensor([[1.0, 0.0]], device="cuda"))
    assert out[0, 0] == 1.0 and out[0, 1].isnan() and out[0, 2] == float("inf") and out[0, 3].isnan()


def test_a_row_named_twice_is_read_twice():
    need_gpu()
    banner("combine the same row twice")
    y = torch.randn(2, 40, device="cuda")
    dest = torch.tensor([[1, 1], [1, 0]], dtype=torch.int32, device="cuda")
    out = mx.expert_combine(y, dest)
    assert torch.equal(out[0], y[1] + y[1]) and torch.equal(out[1], y[1] + y[0])


def test_out_may_be_the_residual_and_padding_stays():
    need_gpu()
    banner("combine in place")
    for dtype in (BF16, F32):
        M, dest, w = routing(19, 2, 4, 0.0, 3)
        y = strided((M, 77), 77, 0, dtype, 1)
        buf = torch.randn(19, 90, device="cuda").to(dtype)
        before = buf.clone()
        want = mx.expert_combine(y, dest, w, residual=before[:, 5:82])
        got = mx.expert_combine(y, dest, w, residual=buf[:, 5:82], out=buf[:, 5:82])
        assert torch.equal(got, want)
        assert torch.equal(buf[:, :5], before[:, :5]) and torch.equal(buf[:, 82:], before[:, 82:])


def test_empty_shapes():
    need_gpu()
    banner("combine empty shapes")
    e = lambda *s: torch.empty(*s, device="cuda")
    dest = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w, r = torch.ones(4, 2, device="cuda"), torch.randn(4, 10, device="cuda")
    assert not mx.expert_combine(e(0, 10), dest, w).any()            # no rows: every slot is outside
    assert torch.equal(mx.expert_combine(e(0, 10), dest, w, residual=r), r)
    dy, dw = mx.expert_combine_backward(r, e(0, 10), dest, w)
    assert dy.shape == (0, 10) and not dw.any()
    dy, dw = mx.expert_combine_backward(e(4, 0), e(3, 0), dest, w)
    assert dy.shape == (3, 0) and not dw.any()
    assert mx.expert_combine(e(3, 0), dest, w).shape == (4, 0)
    assert mx.expert_combine(e(3, 10), dest[:0], w[:0]).shape == (0, 10)
    assert mx.expert_dispatch(e(0, 10), dest[:0]).shape == (0, 10)
    assert mx.expert_dispatch(r, dest, rows_out=0).shape == (0, 10)


def test_offsets_past_32_bits():
    need_gpu()
    rows, C = 530000, 8200                               # 4.3e9 elements
    banner(f"combine {rows} x {C}")
    y = torch.empty(rows, C, dtype=BF16, device="cuda")
    dest = torch.tensor([[rows - 1, 0], [rows - 2, 524287], [262144, 262143]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    picked = torch.randn(6, C, device="cuda", generator=g).to(BF16)
    y[dest.reshape(-1).long()] = picked
    w = torch.ones(3, 2, device="cuda")
    out = mx.expert_combine(y, dest, w)
    assert torch.equal(out, (picked.float().view(3, 2, C).sum(1)).to(BF16))
    dout = torch.randn(3, C, device="cuda", generator=g).to(BF16)
    dy, dw = mx.expert_combine_backward(dout, y, dest, w, out=y)          # in place: each row is read, then written
    assert torch.equal(dy[dest.reshape(-1).long()], dout.repeat_interleave(2, 0))
    ref = (dout.double().repeat_interleave(2, 0) * picked.double()).sum(1).view(3, 2)
    mag = (dout.double().repeat_interleave(2, 0) * picked.double()).abs().sum(1).view(3, 2)
    assert bool(((dw.double() - ref).abs() <= 48 * U * mag).all())
    tail = y[rows - 4096:]
    tail.fill_(1.0)
    for n in (600, 3000):                                # (addresses past 32 bits)
        assert torch.equal(mx.bias_grad(y[rows - n:]), torch.full((C,), float(n), device="cuda"))


# ------------------------------------------------------------------ bias gradient
def bias_tol(ref_mag, M, E, dtype):
    # a lane adds up at most 64 rows (1024 in one go, 16 waves), then 2 steps over lanes and 15
    # over waves, then every fourth tile and the four sums
    return (64 + 17 + M / 256 / 4 + 4) * U * ref_mag + TINY


@pytest.mark.parametrize("N", [1, 5, 8, 255, 513, 1451, 2880])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bias_grad(N, dtype):
    need_gpu()
    for M in (0, 1, 2, 63, 64, 65, 255, 257, 1024, 1025, 1037, 5000):
        banner(f"bias grad M={M} N={N} {dtype}")
        for ld, shift in ((N, 0), (N + 3, 1)):
            x = strided((M, N), ld, shift, dtype, M)
            xd = f64(x)
            ref, mag = xd.sum(0), np.abs(xd).sum(0)
            for out in (F32, BF16):
                got = mx.bias_grad(x, dtype=out)
                assert got.dtype == out and got.shape == (N,)
                rnd = np.abs(ref) * half_step(BF16) * 1.01 if out == BF16 else 0.0
                close(got, ref, bias_tol(mag, M, 1, dtype) + rnd)


@pytest.mark.parametrize("sizes", [[3], [0, 0, 5, 0], [256, 0, 512, 1], [700, 0, 1, 2000, 255, 257], [1] * 300 + [0] * 20,
                                   [0, 0], [5000], [300, 0, 724], [20] * 256])
def test_grouped_bias_grad(sizes):
    need_gpu()
    banner(f"grouped bias grad {sizes[:8]}")
    offsets = torch.tensor(np.cumsum([0] + sizes), dtype=torch.int32, device="cuda")
    for extra in (0, 40):                                # rows past the last group are not read
        for N, dtype in ((100, F32), (1451, BF16), (2880, BF16)):
            M = sum(sizes) + extra
            x = strided((M, N), N, 0, dtype, 7)
            if extra:
                x[sum(sizes):] = NAN
            got = mx.bias_grad(x, offsets)
            assert got.shape == (len(sizes), N)
            ends, xd = np.cumsum([0] + sizes), f64(x)
            ref = np.stack([xd[a:b].sum(0) for a, b in zip(ends, ends[1:])])
            mag = np.stack([np.abs(xd[a:b]).sum(0) for a, b in zip(ends, ends[1:])])
            close(got, ref, bias_tol(mag, M, len(sizes), dtype))


def test_grouped_bias_grad_clamps_offsets():
    need_gpu()
    banner("grouped bias grad offsets past the rows")
    for M in (600, 1600):
        x = torch.ones(M, 33, device="cuda")
        got = mx.bias_grad(x, torch.tensor([-5, 500, 2**31 - 1, 2**31 - 1], dtype=torch.int32, device="cuda"))
        assert torch.equal(got, torch.tensor([500.0, M - 500.0, 0.0], device="cuda")[:, None].expand(3, 33))


def test_grouped_bias_grad_of_offsets_that_decrease():
    """Experts that claim the same rows again name more tiles than there is room for;
    those past it are left out, and nothing past the workspace is read."""
    need_gpu()
    banner("grouped bias grad offsets that decrease")
    x = torch.ones(2000, 33, device="cuda")
    got = mx.bias_grad(x, torch.tensor([0, 2000] * 40 + [0], dtype=torch.int32, device="cuda"))
    assert got.shape == (80, 33)
    assert torch.equal(got[0], torch.full((33,), 2000.0, device="cuda"))
    assert not got[1::2].any()                           # (2000 .. 0: no rows)


# ------------------------------------------------------------------ streams, graphs, repeats
def test_replays_and_another_stream():
    """Captured calls replayed on changed inputs with eager work between, and eager
    calls on another stream, give what eager calls give."""
    need_gpu()
    banner("expert layer captured and replayed")
    T, E, top, C = 3000, 32, 4, 320
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn(T, E, device="cuda", generator=g)
    x = torch.randn(T, C, device="cuda", generator=g).to(BF16)

    def step():
        ids, w = mx.route(logits, top)
        offsets, rows, dest = mx.expert_sort(ids, E)
        xs = mx.expert_dispatch(x, dest)
        y = mx.expert_combine(xs, dest, w, residual=x)
        dy, dw = mx.expert_combine_backward(y, xs, dest, w)
        return ids, w, offsets, rows, dest, y, dy, dw, mx.bias_grad(dy, offsets), mx.route_backward(dw, logits, ids)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        logits.copy_(torch.randn(T, E, device="cuda", generator=g))
        x.copy_(torch.randn(T, C, device="cuda", generator=g).to(BF16))
        graph.replay()
        want = step()
        for a, b in zip(held, want):
            assert torch.equal(a, b), i
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    for a, b in zip(other, want):
        assert torch.equal(a, b)
