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

    def ask(what, lines):
        text = "".join(what + " " + " ".join(str(int(v)) for v in line) + "\n" for line in lines)
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
    for (M, N, tm, tn), n in zip(cases, rule("c", [(M, N, tn) for M, N, _, tn in cases])):
        load = xcd_load(M, N, tm, tn, n)
        assert sum(load) == -(-M // tm) * -(-N // tn)
        assert max(load) - min(load) <= 1, (M, N, tm, tn, load)


def test_wide_products_keep_a_column_tile_on_one_xcd(rule):
    for N, n in zip((128, 129, 400, 1000, 2880, 65536), rule("c", [(64, N, 16) for N in (128, 129, 400, 1000, 2880, 65536)])):
        assert n % 8 == 0 and 0 <= n - -(-N // 16) < 8
    # (with one row tile there is nothing to share)
    assert rule("c", [(32, 400, 16), (1, 400, 16), (33, 400, 16)]) == [25, 25, 32]


ROWS16, TILE, PIPELINE = 0, 1, 2
CUS = 256


@pytest.mark.parametrize("M,N,E,f4,kernel", [
    # narrow outputs fill the chip with small tiles where a 256-column tile would be mostly empty
    (16384, 16, 0, 1, ROWS16), (16384, 16, 0, 0, ROWS16), (4096, 100, 0, 1, ROWS16), (8192, 128, 0, 1, TILE),
    (8192, 256, 0, 1, TILE), (8192, 256, 0, 0, TILE), (16384, 400, 0, 1, PIPELINE), (16384, 400, 0, 0, TILE),
    (16384, 640, 0, 0, PIPELINE), (16384, 16, 32, 1, ROWS16), (16384, 128, 32, 1, TILE), (16384, 128, 8, 0, TILE),
    # one round of 128-row tiles, but not two: row tiles of experts that are mostly full
    (16384, 200, 8, 1, PIPELINE), (16384, 200, 32, 1, PIPELINE), (8192, 400, 8, 1, PIPELINE), (2048, 400, 8, 1, TILE),
    (16384, 400, 32, 0, PIPELINE),
    # wide outputs
    (1, 65536, 0, 1, ROWS16), (32, 11264, 0, 1, ROWS16), (192, 2880, 0, 1, TILE), (1280, 2880, 0, 1, TILE),
    (1400, 2880, 0, 1, PIPELINE), (2048, 2880, 0, 0, TILE), (3000, 2880, 0, 0, PIPELINE), (16384, 2880, 0, 1, PIPELINE),
    (64, 2880, 32, 1, ROWS16), (256, 4096, 8, 1, TILE), (2048, 2048, 4, 1, TILE),
    (1024, 4096, 8, 1, PIPELINE), (768, 2880, 32, 1, PIPELINE),
    (4096, 2880, 32, 0, TILE), (8192, 2880, 32, 0, PIPELINE), (65536, 2880, 32, 1, PIPELINE)])
def test_kernel(rule, M, N, E, f4, kernel):
    """On 256 CUs, MXFP4 or MXFP8: the faster kernel of those measured beside the rule."""
    assert rule("k", [(M, N, E, f4, not f4, CUS)]) == [kernel]


def test_waves(rule):
    sizes = [(1, 2880, 0), (64, 2880, 0), (128, 2880, 0), (64, 2880, 32), (8192, 16, 0), (16384, 16, 0)]
    assert rule("w", [(*s, CUS) for s in sizes]) == [8, 4, 2, 2, 8, 4]
