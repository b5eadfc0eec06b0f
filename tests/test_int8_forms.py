"""Forms of the 8-bit integer linear that are not built (no GPU): the plan never chooses one, by the same rule by which the
launcher refuses it, so that no call returns without having launched."""
import math
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "int8_plan.h"
using mbq::Int8Form;
static_assert(!mbq::serves_int8(Int8Form::kStream8x1, 0, false), "one weight's codes have no form of 8 waves");
static_assert(mbq::serves_int8(Int8Form::kStream8x1, 0, true) && mbq::serves_int8(Int8Form::kStream8x1, 1, false));
static_assert(mbq::serves_int8(Int8Form::kStream16x1, 0, false) && mbq::serves_int8(Int8Form::kShared256x256, 0, false));
int main() {
  int t, p, n, k, gated, experts, codes, streams = 0;
  while (std::scanf("%d %d %d %d %d %d %d", &t, &p, &n, &k, &gated, &experts, &codes) == 7) {
    const mbq::Int8Plan q = mbq::plan_int8(t, p, experts, (n + 15) / 16, gated + 1, (k + 127) / 128, codes);
    if (!mbq::serves_int8(q.form, experts, q.inline_x)) return 1;
    streams += q.form == Int8Form::kStream8x1 || q.form == Int8Form::kStream16x1;
  }
  std::printf("%d\n", streams);
  return 0;
}
"""


def test_no_plan_has_a_form_that_is_not_built(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    (tmp_path / "forms.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "token_adaptive_bit_amd", "csrc"),
                    str(tmp_path / "forms.cpp"), "-o", str(tmp_path / "forms")], check=True)
    rng = random.Random(5)
    cases = []
    for _ in range(20000):                                   # few tokens above all: there streaming forms are chosen
        experts = rng.choice([0, 0, 1, rng.randint(2, 300)])
        t = int(round(math.exp(rng.uniform(0, math.log(rng.choice([16, 16, 4096]))))))
        n, k = (int(round(math.exp(rng.uniform(0, math.log(hi))))) for hi in (1 << 17, (1 << 17) - 1))
        cases.append((t, t if not experts else t * rng.randint(1, 8), n, k, rng.randint(0, 1), experts, rng.randint(0, 1)))
    res = subprocess.run([str(tmp_path / "forms")], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True)
    assert res.returncode == 0
    assert int(res.stdout) > 1000                            # of 20000: the rule was asked where it matters
