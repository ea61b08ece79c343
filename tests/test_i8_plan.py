"""Which tile, how many splits of K and which way of reading the weights each case of
tests/test_gpu_i8_tiles.py takes: together they launch every tile of the 8-bit products. The
plan is host code; it is compiled here on its own (no GPU)."""
import os
import shutil
import subprocess

import pytest

from sparse_expert_ffn_amd import buildlib
from tests.test_ffn_asm_hazards import HIPCC

# rows x columns of a tile, as ffn_plan.h numbers them
T256, T128, T64, T16, T256X128 = range(5)

# (S, K, N): (tile, K is split, one row of tiles). Sizes off the tiles; K off the stages of 128
MATMUL = {
    (5465, 656, 5720): (T256, False, False), (445, 6288, 5504): (T256, True, False),
    (764, 928, 2712): (T128, False, False), (67, 4624, 5656): (T128, True, True),
    (1001, 2064, 776): (T64, False, False), (53, 784, 9160): (T64, False, True),
    (317, 3344, 24): (T64, True, False), (17, 6000, 1352): (T64, True, True),
    (33, 1040, 200): (T16, False, False), (23, 1696, 40): (T16, True, False),
    (16, 8208, 24): (T16, True, True), (11, 80, 16392): (T16, False, True),
    (3411, 272, 1208): (T256X128, False, False), (5553, 3344, 24): (T256X128, True, False),
    (168, 6032, 5592): (T256X128, True, True),
}
# (S, H, D): those of up and gate in one product. D above 8192 takes the general join where K is
# split and more threads to a row in h's quantisation; up to it one launch joins and quantises
FFN = {
    (5464, 656, 5712): (T256, False, False), (177, 7696, 6240): (T256, True, True),
    (576, 4192, 2496): (T128, False, False), (65, 1120, 8880): (T128, False, True),
    (69, 5984, 2736): (T128, True, True), (1001, 2064, 784): (T64, False, False),
    (37, 144, 11504): (T64, False, True), (415, 2528, 16): (T64, True, False),
    (27, 6624, 1632): (T64, True, True), (64, 7168, 2064): (T64, True, True),
    (17, 48, 64): (T16, False, False), (20, 1936, 80): (T16, True, False),
    (5, 64, 16400): (T16, False, True), (13, 4112, 8176): (T16, True, True),
    (16, 8192, 8208): (T16, True, True), (5, 80, 131072): (T16, False, True),
    (764, 928, 2704): (T256X128, False, False), (135, 336, 11536): (T256X128, False, True),
    (142, 6000, 3024): (T256X128, True, True),
}

SOURCE = r"""
#include <cstdio>
#include "ffn_plan.h"
int main() {
  long dual, M, N, K;
  while (std::scanf("%ld %ld %ld %ld", &dual, &M, &N, &K) == 4) {
    const moe::GemmPlan p = moe::plan_gemm(moe::kPlanI8, 31u, dual != 0, M, N, K, 1);
    std::printf("%d %d %d\n", p.tile, p.splits, p.tiles_m);
  }
}
"""


@pytest.mark.skipif(shutil.which(HIPCC) is None, reason="hipcc not available")
def test_every_tile_has_a_case(tmp_path):
    src, exe = tmp_path / "plan.hip", tmp_path / "plan"
    src.write_text(SOURCE)
    csrc = os.path.join(buildlib.PKG, "csrc")
    r = subprocess.run([HIPCC, f"--offload-arch={buildlib.ARCH}", "-std=c++17", "--cuda-host-only",
                        "-I", os.path.join(buildlib.ROOT, "include"), "-I", csrc, "-I",
                        os.path.join(csrc, "ffn"), str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    asked = [(0, S, N, K) for S, K, N in MATMUL] + [(1, S, D, H) for S, H, D in FFN]
    r = subprocess.run([str(exe)], input="".join("%d %d %d %d\n" % a for a in asked),
                       capture_output=True, text=True, check=True)
    got = [(int(t), int(s) > 1, int(m) == 1) for t, s, m in map(str.split, r.stdout.splitlines())]
    want = list(MATMUL.values()) + list(FFN.values())
    assert len(got) == len(want)
    wrong = [(a, g, w) for a, g, w in zip(asked, got, want) if g != w]
    assert not wrong, wrong
    for cases in (MATMUL, FFN):
        assert {t for t, _, _ in cases.values()} == set(range(5))
        # the two small tiles have a kernel of their own for weights that are read once
        assert {(t, s, o) for t, s, o in cases.values() if t in (T64, T16)} == {
            (t, s, o) for t in (T64, T16) for s in (False, True) for o in (False, True)}
