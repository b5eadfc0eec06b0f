"""The plan of the 8-bit integer linear (no GPU): csrc/int8_plan.h compiled by itself, and the shapes that the GPU tests
run its forms on."""
import math
import os
import random
import shutil
import subprocess

import pytest

from int8_paths import FORMS, PATHS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "int8_plan.h"
// t p n k gated experts codes -> form chunks inline, and what the kernels need of them
int main() {
  int t, p, n, k, gated, experts, codes;
  while (std::scanf("%d %d %d %d %d %d %d", &t, &p, &n, &k, &gated, &experts, &codes) == 7) {
    const int groups = (n + 15) / 16, kb = (k + 127) / 128;
    const mbq::Int8Plan q = mbq::plan_int8(t, p, experts, groups, gated + 1, kb, codes);
    const int form = int(q.form), per = (kb + q.chunks - 1) / q.chunks;
    const mbq::Int8Cost& c = mbq::kInt8Costs[form];
    if (form < 0 || form >= mbq::kInt8Forms) return 1;
    if (q.chunks < 1 || (q.chunks - 1) * per >= kb || q.chunks * per < kb) return 2;  // an empty chunk, or blocks left over
    if (q.chunks > 1 && (experts || form < 3)) return 3;                            // K is split for one weight's tiles
    if (form < 3 && !experts && t > c.tokens) return 4;                             // a streaming workgroup's tokens
    if (form < 3 && experts && p / 16 + experts > 65535) return 5;                  // its grid
    if (q.inline_x && (codes || form > 1 || long(p < 16 ? p : 16) * kb > mbq::kInt8Inline)) return 6;
    const long tiles = long((groups * (gated + 1) * 16 + c.rows - 1) / c.rows) * ((t + c.tokens - 1) / c.tokens) * q.chunks;
    const int left = tiles % 256;
    const int cut = form < 9 || experts ? 0 : tiles < 256 || left == 0 || left > 128 ? 1 : left > 64 ? 2 : 4;
    std::printf("%d %d %d %d\n", form, int(q.chunks > 1), int(q.inline_x), cut);
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("int8_plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I",
                    os.path.join(ROOT, "token_adaptive_bit_amd", "csrc"), str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def run(cases):
        res = subprocess.run([str(d / "plan")], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True)
        assert res.returncode == 0, (res.returncode, res.stderr[-500:])
        out = res.stdout.splitlines()
        assert len(out) == len(cases)
        return [tuple(map(int, line.split())) for line in out]
    return run


def test_every_shape_has_its_form(plan):
    keys = list(PATHS)
    got = plan([(t, p, n, k, key[0], experts, codes) for key, (t, p, n, k, experts, codes) in PATHS.items()])
    assert got == [key[2:] for key in keys]
    for gated in (0, 1):
        assert {k[2] for k in keys if k[0] == gated} == set(range(len(FORMS)))


def test_every_choice_can_be_launched(plan):
    """Whatever the sizes: chunks that cover K with none empty, grids and LDS within their limits."""
    rng = random.Random(0)

    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    cases = []
    for _ in range(20000):
        experts = rng.choice([0, 0, 1, log_int(1, 1024)])
        t = log_int(1, 1 << 21)
        cases.append((t, t if not experts else log_int(1, 1 << 24), log_int(1, 1 << 20), log_int(1, (1 << 17) - 1), rng.randint(0, 1),
                      experts, rng.randint(0, 1)))
    plan(cases)
