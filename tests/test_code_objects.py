"""What the compiler made of the MXFP8 / MXFP6 pipeline's kernels: no spills, and output
buffers held to be the same in every lane.  (Where it cannot tell, every store stands in a
loop that reads the buffer's words from the first lane and compares: hundreds of
v_readfirstlane in a kernel that otherwise has a few dozen, the plain products 3-5 %
slower.)"""
import os
import re

import pytest

import mxfp4_microscaling_quantization_mx_amd as mx

FAMILIES = ("k_gemm_f8", "k_gemm_f8_q", "k_grouped_gemm_f8", "k_grouped_gemm_f8_q", "k_gated_f8", "k_grouped_gated_f8",
            "k_linear_f8", "k_grouped_linear_f8")


@pytest.fixture(scope="module")
def objects():
    pytest.importorskip("msgpack")
    import code_objects as co
    if not os.path.exists(mx.LIB_PATH) or not os.path.exists(co.OBJDUMP):
        pytest.skip("libmxfp4.so not built, or no disassembler")
    return [(elf, co.kernels(elf)) for elf in co.code_objects(mx.LIB_PATH)]


def of_family(family, names):
    return sorted(n for n in names if re.search(r"\d%sI" % family, n))


@pytest.mark.parametrize("family", FAMILIES)
def test_no_spills(objects, family):
    """FP6 A with FP8 B of the dense quantizing epilogue keeps two registers in scratch."""
    found = {n: k for _, ks in objects for n, k in ks.items() if n in of_family(family, ks)}
    assert found
    for name, k in found.items():
        allowed = 2 if re.search(r"\dk_gemm_f8_qILi[34]ELi[12]E", name) else 0
        assert k[".vgpr_spill_count"] <= allowed, name
        assert allowed or k[".private_segment_fixed_size"] == 0, name


@pytest.mark.parametrize("family", FAMILIES)
def test_output_buffers_are_uniform(objects, family, tmp_path):
    import code_objects as co
    for i, (elf, ks) in enumerate(objects):
        names = of_family(family, ks)[:2]
        if not names:
            continue
        path = tmp_path / f"{i}.co"
        path.write_bytes(elf)
        for name, code in co.instructions(str(path), names).items():
            count = sum(m.startswith("v_readfirstlane") for m in code)
            stores = sum(m.startswith("buffer_store") for m in code)
            assert stores and count < 150, (name, count, stores)


def test_the_gated_block_takes_its_own_arguments(objects):
    """Kernels that share a body do not share the linear layer's arguments (with them the gated
    block's 128-row tiles took 1-3 % longer)."""
    size = {n: k[".kernarg_segment_size"] for _, ks in objects for n, k in ks.items()}
    linear = {size[n] for n in of_family("k_linear_tile", size)}
    gated = {size[n] for f in ("k_gated_tile", "k_gated_few") for n in of_family(f, size)}
    assert linear and gated and max(gated) < min(linear)
