"""Sizes that the library refuses reach it: the binding does not allocate outputs of them
first (here an allocation fails the test)."""
import pytest
import torch

import mxfp4_microscaling_quantization_mx_amd as mx
from test_binding_devices_experts import on


@pytest.fixture(autouse=True)
def stream(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.mark.parametrize("status,f", [
    (mx.MX_ERR_UNSUPPORTED, lambda: mx.expert_sort(on(i32(4, 2), 0), 1 << 60)),
    (mx.MX_ERR_UNSUPPORTED, lambda: mx.expert_sort(on(i32(4, 2), 0), 2000000000)),
    (mx.MX_ERR_UNSUPPORTED, lambda: mx.expert_sort(on(i32(4, 2), 0), (1 << 32) + 32)),
    (mx.MX_ERR_INVALID_ARG, lambda: mx.expert_sort(on(i32(4, 2), 0), -1)),
    (mx.MX_ERR_INVALID_ARG, lambda: mx.expert_sort(on(i32(4, 2), 0), -(1 << 40))),
    (mx.MX_ERR_INVALID_ARG, lambda: mx.route(on(torch.zeros(4, 8), 0), 1 << 60)),
    (mx.MX_ERR_INVALID_ARG, lambda: mx.route(on(torch.zeros(4, 8), 0), 1 << 29)),
    (mx.MX_ERR_INVALID_ARG, lambda: mx.route(on(torch.zeros(4, 8), 0), 0)),
    (mx.MX_ERR_INVALID_ARG, lambda: mx.route(on(torch.zeros(4, 8), 0), -3)),
])
def test_refused_sizes_are_not_allocated(status, f):
    with pytest.raises(mx.MXError) as e:
        f()
    assert e.value.status == status
