"""The host rule that picks the dense MXFP4 product's kernel and cuts it, built with the undefined-behaviour checks of
the host compiler: no size a call may have divides by zero or overflows, and every plan covers its product."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_latent_moe_amd", "csrc")
MAIN = r"""
#include <cstdio>
#include "mx4_plan.h"
int main() {
  int T, N, K;
  while (std::scanf("%d %d %d", &T, &N, &K) == 3) {
    const moe::Mx4Plan p = moe::mx4_plan(T, N, K);
    std::printf("%zu %d %d %d %d\n", moe::mx4_partial_bytes(T, N, K), (int)p.stream, p.rows, p.cut, p.splits);
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


SIZES = [(T, N, K) for T in (0, 1, 16, 17, 64, 65, 300, 4096, 1 << 21) for N in (1, 127, 895, 6144, 1 << 20)
         for K in (32, 416, 7168, 33792, 1 << 20) if T * N <= 1 << 33]  # what a call may have


def test_every_plan_covers_its_product(plan):
    up = lambda a, b: -(-a // b)  # noqa: E731
    for (T, N, K), (need, stream, rows, cut, splits) in zip(SIZES, plan(SIZES)):
        assert stream or T > 16
        assert need == (splits * T * up(N, 4) * 16 if splits > 1 else 0)
        if stream:
            assert (rows, cut, splits) == (0, 0, 1)
            groups = up(N, 32) * up(T, 64)
        else:
            assert rows in (64, 128, 192, 256) and 0 <= cut < up(N, 256)
            assert 1 <= splits <= up(K, 512) and (splits == 1 or cut == 0)
            groups = cut * up(T, 256) + (up(N, 256) - cut) * up(T, rows) * splits + 16
        assert groups * 512 < 2 ** 32  # the threads of one grid


def test_sizes_of_the_product_tests(plan):
    """The sizes with which the GPU tests mean to reach every kind of cut."""
    kinds = set()
    for _, stream, rows, cut, splits in plan([(301, 895, 7168), (512, 3584, 7168), (1500, 2100, 256),
                                              (2900, 4400, 1056), (4100, 6200, 768), (3000, 6600, 1536),
                                              (4096, 4096, 4096)]):
        kinds.add("stream" if stream else f"{rows} {'cut' if cut else 'parts' if splits > 1 else 'whole'}")
    assert kinds == {"stream", "64 parts", "64 whole", "128 whole", "192 cut", "64 cut", "256 whole"}
