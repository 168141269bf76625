"""Plain 64-bit forms of the expert layer's operators for its tests (NumPy on
the host; nothing of the library is used)."""
import numpy as np
import torch

U = 2.0 ** -24                       # half a float32 step at 1
TINY = 2.0 ** -120                   # far above the smallest normal number, where a result may be flushed


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def choose(logits, top):
    """Largest first, ties to the lowest index, NaN above every number."""
    out = np.empty((logits.shape[0], top), np.int32)
    for t, row in enumerate(logits):
        key = [(0 if np.isnan(v) else 1, 0.0 if np.isnan(v) else -v, e) for e, v in enumerate(row)]
        out[t] = [k[2] for k in sorted(key)[:top]]
    return out


def _softmax(x):
    """Rows whose largest is -Inf: zeros."""
    with np.errstate(all="ignore"):
        m = x.max(1, keepdims=True)
        e = np.exp(x - m)
        p = e / e.sum(1, keepdims=True)
    return np.where(m == -np.inf, 0.0, p)


def scores(logits, score):
    with np.errstate(all="ignore"):
        return _softmax(logits) if score == "softmax" else 1 / (1 + np.exp(-logits))


def weights(logits, ids, score, renorm):
    """Routing weights at scale 1."""
    chosen = np.take_along_axis(logits, ids, 1)
    if score == "softmax":
        return _softmax(chosen) if renorm else np.take_along_axis(_softmax(logits), ids, 1)
    with np.errstate(all="ignore"):
        if not renorm:
            return 1 / (1 + np.exp(-chosen))
        return _softmax(-np.logaddexp(0, -chosen))      # log s = -log(1 + e^-l)


def weight_bound(logits, ids, score, E):
    """The relative error that include/mx.h allows a weight."""
    chosen = np.take_along_axis(logits, ids, 1)
    with np.errstate(all="ignore"):
        d = np.nanmax(np.where(np.isinf(chosen), np.nan, chosen), 1, initial=-1e30, keepdims=True) - chosen
    d = np.where(np.isfinite(d), np.abs(d), 0.0)
    return (32 + np.log(E) + d) * U


def sort_slots(ids, E):
    T, top = ids.shape
    flat = ids.reshape(-1)
    order = np.concatenate([np.flatnonzero(flat == e) for e in range(E)] + [np.empty(0, np.int64)]).astype(np.int64)
    rows, dest = np.full(T * top, -1, np.int32), np.full(T * top, -1, np.int32)
    rows[:order.size] = order // top
    dest[order] = np.arange(order.size)
    offsets = np.cumsum([0] + [np.count_nonzero(flat == e) for e in range(E)]).astype(np.int32)
    return offsets, rows, dest.reshape(T, top)


def strided(shape, ld, shift, dtype, seed=0, std=1.0):
    """A [R, C] tensor of normal values with row stride ld, `shift` elements into
    its storage, whose padding holds NaN."""
    R, C = shape
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((shift + max(R, 1) * ld + 8,), float("nan"), dtype=dtype)
    t = buf.cuda()[shift:shift + max(R, 1) * ld].view(max(R, 1), ld)[:R, :C]
    t.copy_((torch.randn(R, C, generator=g) * std).to(dtype))
    return t
