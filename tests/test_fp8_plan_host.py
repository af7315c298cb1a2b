"""The host rule that picks the 8-bit product's kernel and cuts it, built with the undefined-behaviour checks of the
host compiler: no size a call may have divides by zero or overflows, and every plan covers its product."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_latent_moe_amd", "csrc")
MAIN = r"""
#include <cstdio>
#include "fp8_plan.h"
int main() {
  int T, N, K;
  while (std::scanf("%d %d %d", &T, &N, &K) == 3) {
    std::printf("%zu", moe::fp8_partial_bytes(T, N, K));
    for (bool bf16 : {false, true}) {
      const moe::Fp8Plan p = moe::fp8_plan(T, N, K, bf16);
      std::printf(" %d %d %d", (int)p.stream, p.stream ? 0 : p.tile.rows, p.stream ? 1 : p.tile.splits);
    }
    std::printf("\n");
    std::fflush(stdout);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC,
                    str(d / "main.cpp"), "-o", str(d / "plan")], check=True)

    def run(sizes):
        r = subprocess.run([str(d / "plan")], input="".join("%d %d %d\n" % s for s in sizes), capture_output=True,
                           text=True)
        assert r.returncode == 0, f"{sizes[len(r.stdout.splitlines())]}: {r.stderr}"
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]

    return run


BIG = 1 << 22
SIZES = [(T, N, K) for T in (0, 1, 64, 65, 300, 4096, BIG) for N in (1, 127, 895, 6144, BIG)
         for K in (16, 400, 7168, 1 << 20)]


def test_every_plan_covers_its_product(plan):
    for (T, N, K), (need, *p) in zip(SIZES, plan(SIZES)):
        kb, most = -(-K // 128), 0
        for bf16, (stream, rows, splits) in enumerate((p[:3], p[3:])):
            assert stream or T > 64
            assert rows % 256 == 0 and (bf16 or rows == 0) and (rows - N < 256)
            assert 1 <= splits <= max(1, kb // 4) and (splits == 1 or rows == 0)
            if splits > 1:
                most = max(most, splits * T * -(-N // 4) * 16)
        assert need == most


def test_no_tokens_need_no_plan(plan):
    assert plan([(0, 3584, 7168)]) == [(0, 1, 0, 1, 1, 0, 1)]


def test_sizes_of_the_parts_tests(plan):
    """The sizes with which the GPU tests mean to split K, in both outputs."""
    for need, s32, _, k32, s16, _, k16 in plan([(301, 895, 7168), (301, 893, 7168), (130, 3002, 4112)]):
        assert not s32 and not s16 and k32 > 1 and k16 > 1 and need > 0
