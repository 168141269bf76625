"""How the products with a float32 epilogue are cut into workgroups (csrc/launch_rule.h,
compiled for the host)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mxfp4_microscaling_quantization_mx_amd", "csrc")


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("rule") / "rule")
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, os.path.join(HERE, "launch_rule.cpp"), "-o", exe], check=True)

    def ask(lines):
        text = "".join(" ".join(str(int(v)) for v in line) + "\n" for line in lines)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
        assert len(out) == len(lines)
        return [int(v) for v in out]
    return ask


def xcd_load(M, N, tm, tn, padded):
    """Real tiles on each of 8 XCDs, workgroup b on XCD b % 8."""
    load, real = [0] * 8, -(-N // tn)
    for t in range(padded * -(-M // tm)):
        load[t % 8] += t % padded < real
    return load


def test_narrow_products_use_every_xcd(rule):
    cases = [(M, N, tm, tn) for tm, tn in ((16, 16), (32, 16), (128, 128), (128, 64)) for M in (2048, 8192)
             for N in (1, tn - 1, tn, tn + 1, 3 * tn, 7 * tn)]
    for (M, N, tm, tn), n in zip(cases, rule([(M, N, tn) for M, N, _, tn in cases])):
        load = xcd_load(M, N, tm, tn, n)
        assert sum(load) == -(-M // tm) * -(-N // tn)
        assert max(load) - min(load) <= 1, (M, N, tm, tn, load)


def test_wide_products_keep_a_column_tile_on_one_xcd(rule):
    for N, n in zip((128, 129, 400, 1000, 2880, 65536), rule([(64, N, 16) for N in (128, 129, 400, 1000, 2880, 65536)])):
        assert n % 8 == 0 and 0 <= n - -(-N // 16) < 8
    # (with one row tile there is nothing to share)
    assert rule([(32, 400, 16), (1, 400, 16), (33, 400, 16)]) == [25, 25, 32]
