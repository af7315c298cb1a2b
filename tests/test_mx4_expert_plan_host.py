"""The host rules of the expert products on MXFP4 rows, and which kernels the sizes of test_gpu_mx4_direct.py reach:
csrc/mx4_plan.h built with the undefined-behaviour checks of the host compiler."""
import os
import shutil
import subprocess

import pytest
from test_gpu_mx4_direct import DENSE, EXPERTS, LONG
from test_gpu_mx4_layer_lists import BOTH, TILES, WIDE

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_latent_moe_amd", "csrc")
MAIN = r"""
#include <cstdio>
#include "mx4_plan.h"
using namespace moe;
int main() {
  char kind;
  int a, b, c;
  while (std::scanf(" %c %d %d %d", &kind, &a, &b, &c) == 4) {
    if (kind == 'd') {
      const Mx4Plan p = mx4_plan(a, b, c);
      std::printf("%d %d %d %d\n", (int)p.stream, p.rows, p.cut, p.splits);
    } else {
      const int groups = mx4_stream_groups(c, kind == 'p');
      std::printf("%d %d %d %d %d %d\n", (int)mx4_finds_chunks(a, b, groups), mx4_found_chunks(a, b), groups,
                  mx4_few_rows(a, b), mx4_few_chunks(a, b), mx4_many_chunks(a, b));
    }
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

    def run(kind, sizes):
        r = subprocess.run([str(d / "plan")], input="".join("%s %d %d %d\n" % (kind, *s) for s in sizes),
                           capture_output=True, text=True)
        assert r.returncode == 0, f"{sizes[len(r.stdout.splitlines())]}: {r.stderr}"
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]

    return run


def test_dense_sizes(plan):
    kinds = set()
    for (T, _, K), (stream, rows, cut, splits) in zip(DENSE, plan("d", DENSE)):
        assert K % 128 == 0
        kinds.add(f"stream {16 if T <= 16 else 32 if T <= 32 else 64}" if stream
                  else f"{rows} {'cut' if cut else 'parts' if splits > 1 else 'whole'}")
    assert kinds == {"stream 16", "stream 32", "stream 64", "64 whole", "64 parts", "64 cut", "128 whole", "128 parts",
                     "192 whole", "192 cut", "256 whole"}
    [(stream, rows, _, splits)] = plan("d", [LONG])
    assert not stream and rows == 256 and splits > 1


def chunk_rows(counts, few):
    """Rows of the chunks: blocks of 64 shared evenly over as few chunks of 256 as there can be."""
    for n in counts:
        if n > few:
            blocks, parts = -(-n // 64), -(-n // 256)
            for i in range(parts):
                yield min(64 * (blocks * (i + 1) // parts), n) - 64 * (blocks * i // parts)


def test_expert_sizes(plan):
    """The counts reach the kernels that their names say, tiles of every height among them."""
    heights = set()
    for name, (counts, inter, latent) in EXPERTS.items():
        for kind, N in (("p", inter), ("s", latent)):
            [(finds, _, _, few, _, many)] = plan(kind, [(len(counts), sum(counts) + 3, N)])
            if name == "found":
                assert finds
                continue
            assert not finds and many > 0
            small, large = any(0 < n <= few for n in counts), any(n > few for n in counts)
            assert (few == 0, small, large) == {"tiles": (True, False, True), "both": (False, True, True),
                                                "streamed": (False, True, False)}[name]
            heights |= {-(-n // 64) for n in chunk_rows(counts, few)}
    assert heights == {1, 2, 3, 4}


def test_lists_hold_every_chunk(plan):
    """For any spread of P rows over E experts: no more chunks than the lists have room for, and grids of fewer than
    2^32 threads."""
    sizes = [(E, P, N) for E in (1, 2, 7, 64, 896, 1024) for P in (1, 16, 17, 31, 300, 5000, 65536, 1 << 21)
             for N in (1, 64, 3584, 1 << 18) if P * N <= 1 << 33]
    for kind in "ps":
        for (E, P, N), (finds, found, groups, few, few_cap, many_cap) in zip(sizes, plan(kind, sizes)):
            spreads = [[P], [P // E] * E, [1] * min(E, P), [17] * min(E, P // 17), [16] * min(E, P // 16),
                       [257] * min(E, P // 257)]
            for counts in spreads:
                spare = P - sum(counts)
                for c in ([*counts[:-1], counts[-1] + spare] if counts else [P], counts):
                    assert sum(-(-n // 64) for n in c) <= found
                    assert sum(0 < n <= few for n in c) <= few_cap
                    assert sum(-(-n // 256) for n in c if n > few) <= many_cap
            assert groups * (found if finds else few_cap) * 256 < 2 ** 32
            assert -(-N // (128 if kind == "p" else 256)) * many_cap * 512 < 2 ** 32


def test_layer_sizes(plan):
    """The layer test's token counts: lists for both products, on either side of 32 rows an expert."""
    for T, few in ((BOTH, 16), (TILES, 0)):
        for kind, N in (("p", WIDE.inter), ("s", WIDE.latent)):
            [(finds, _, _, few_rows, _, many)] = plan(kind, [(WIDE.n_experts, T * WIDE.top_k, N)])
            assert not finds and few_rows == few and many > 0
