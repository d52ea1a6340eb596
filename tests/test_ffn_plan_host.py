"""Which kernel and how many tiles the sizes of the tests reach: the library's own
choice, from its object files linked with a small entry point."""
import ctypes
import os
import subprocess

import pytest

from decode_projection_gemms_gb300 import build as b
from ffn_cases import MANY_ROUNDS

SMS = 152

SOURCE = """
#include "kp_ffn.cuh"
extern "C" __attribute__((visibility("default"))) int uses_tile(int mx4, int gated, int M, int N, int K, int sms) {
    return kp::ffn_use_tile(mx4, gated, M, N, K, sms);
}
"""


@pytest.fixture(scope="module")
def uses_tile(tmp_path_factory):
    objects = [os.path.join(b.BUILD, os.path.splitext(s)[0] + ".o") for s in b.SOURCES]
    b.build(force=not all(os.path.exists(o) for o in objects))
    d = tmp_path_factory.mktemp("plan")
    src, out = str(d / "plan.cu"), str(d / "plan.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([b.nvcc(), *b.NVCC_FLAGS, "-I", b.CSRC, "-shared", "-o", out, src, *objects], check=True)
    return ctypes.CDLL(out).uses_tile


@pytest.mark.parametrize("mx4,gated,T,F,K", MANY_ROUNDS)
def test_many_rounds_take_the_tile_kernel(uses_tile, mx4, gated, T, F, K):
    assert uses_tile(mx4, gated, T, F, K, SMS) == 1
    # tiles are 256 rows by at most 256 accumulator columns, half of them outputs in
    # the gated forms; an SM pair works on one
    tiles = -(-T // 256) * -(-F // (128 if gated else 256))
    assert tiles > 2 * (SMS // 2)
    assert -(-K // (256 if mx4 else 64)) > 8


def test_few_tokens_do_not(uses_tile):
    assert uses_tile(0, 1, 1, 2048, 7168, SMS) == 0 and uses_tile(1, 0, 8, 4096, 7168, SMS) == 0
