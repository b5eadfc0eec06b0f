"""The plan of the 8-bit linear (no GPU): csrc/fp8_plan.h compiled by itself, and the shapes
that the GPU tests run its forms on."""
import math
import os
import random
import shutil
import subprocess

import pytest

from fp8_paths import STREAMS, TILES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "fp8_plan.h"
// t n k gated exact -> "stream waves token_tiles" or "tile tile split"
int main() {
  int t, n, k, gated, exact;
  while (std::scanf("%d %d %d %d %d", &t, &n, &k, &gated, &exact) == 5) {
    const int groups = (n + 15) / 16, kb = (k + 127) / 128;
    if (mbq::streams(t, groups, kb)) {
      const mbq::StreamPlan p = mbq::plan_stream(t, groups, kb);
      std::printf("stream %d %d\n", p.waves, p.token_tiles);
    } else {
      const mbq::Plan p = mbq::plan_gemm(t, groups * (gated + 1), kb, exact);
      const int per = (kb + p.chunks - 1) / p.chunks;
      if (p.chunks < 1 || (p.chunks - 1) * per >= kb || p.chunks * per < kb) return 1;  // an empty chunk, or blocks left over
      std::printf("tile %d %d\n", p.tile, p.chunks > 1);
    }
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def paths(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "token_adaptive_bit_amd", "csrc"), str(d / "plan.cpp"),
                    "-o", str(d / "plan")], check=True)

    def run(cases):
        out = subprocess.run([str(d / "plan")], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True,
                             text=True, check=True).stdout.splitlines()
        assert len(out) == len(cases)
        return [(kind, int(a), int(b)) for kind, a, b in (line.split() for line in out)]
    return run


def test_every_shape_has_its_form(paths):
    keys = list(TILES)
    got = paths([(*TILES[k], k[0], k[1]) for k in keys])
    assert got == [("tile", tile, split) for _, _, tile, split in keys]
    keys = list(STREAMS)
    assert paths([(*STREAMS[k], k[0], 0) for k in keys]) == [("stream", waves, tiles) for _, waves, tiles in keys]


def test_no_other_form_is_chosen(paths):
    """Shapes over the whole range choose the forms of the tables, and all of them."""
    rng = random.Random(0)

    def draw(lo, hi):
        return int(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    cases = [(draw(1, 1 << 15), draw(1, 1 << 17), draw(1, 1 << 16), rng.randrange(2), rng.randrange(2)) for _ in range(200000)]
    tiles, streams = set(), set()
    for (_, _, _, gated, exact), (kind, a, b) in zip(cases, paths(cases)):
        (streams if kind == "stream" else tiles).add((gated, a, b) if kind == "stream" else (gated, exact, a, b))
    assert tiles == set(TILES) and streams == set(STREAMS)
