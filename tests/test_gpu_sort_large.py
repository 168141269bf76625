"""The sort by expert at sizes whose running sums take several steps of 64 chunks."""
import numpy as np
import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx
from gpu_util import banner, host, need_gpu

pytestmark = pytest.mark.gpu


def stable(ids, E):
    """offsets, rows and dest from numpy's stable sort."""
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(key, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])]).astype(np.int32)
    order = order[:offsets[E]]
    rows, dest = np.full(flat.size, -1, np.int32), np.full(flat.size, -1, np.int32)
    rows[:order.size] = order // ids.shape[1]
    dest[order] = np.arange(order.size)
    return offsets, rows, dest.reshape(ids.shape)


@pytest.mark.parametrize("T,top,E", [(262144, 4, 256), (1048577, 1, 1024), (131073, 8, 7)])
def test_sort_of_a_million_slots(T, top, E):
    """256 chunks and one more, skewed and with dropped ids."""
    need_gpu()
    banner(f"sort T={T} top={top} E={E}")
    g = np.random.default_rng([T, E])
    ids = (g.random((T, top)) ** 3 * E).astype(np.int32)
    drop = g.random((T, top)) < 0.05
    ids = np.where(drop, g.choice([-1, E, -2**31, 2**31 - 1], (T, top)), ids).astype(np.int32)
    dev = torch.from_numpy(ids).cuda()
    want = stable(ids, E)
    for _ in range(2):
        for got, ref, name in zip(mx.expert_sort(dev, E), want, ("offsets", "rows", "dest")):
            assert np.array_equal(host(got), ref), name
