"""The slope of the SiLU's sigmoid is looked at for the SiLU alone, as include/mx.h says."""
import os

import pytest

import mxfp4_microscaling_quantization_mx_amd as mx
from test_abi_linear import BAD, CALLS, OK, _cfg, _tensor, call

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mx.LIB_PATH):
        pytest.skip("libmxfp4.so not built")
    return mx.load_library()


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("alpha", [0.0, -1.0, NAN, INF])
def test_alpha_is_the_silus(lib, name, alpha):
    none = dict(a=_tensor(0, 96))              # (no rows: checked, and nothing launched)
    for act in (1, 2, 3):
        if act == 3 and "backward" in name:
            continue
        assert call(lib, name, cfg=_cfg(act, alpha), **none) == (OK, b"")
    assert call(lib, name, cfg=_cfg(0, alpha), **none)[0] == BAD
