"""The shapes of tests/expert_tails.py (no GPU): the plan chooses their form, their tiles pass a round of the units, and the
last part round is dealt as their key says, with tiles that leave parts without tokens and tiles that end inside 16."""
import os
import shutil
import subprocess

import pytest

from expert_tails import TAILS, TILES, UNITS, counts, tiles

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "int8_plan.h"
int main() {
  int t, p, n, k, gated, experts, codes;
  while (std::scanf("%d %d %d %d %d %d %d", &t, &p, &n, &k, &gated, &experts, &codes) == 7)
    std::printf("%d\n", int(mbq::plan_int8(t, p, experts, (n + 15) / 16, gated + 1, (k + 127) / 128, codes).form));
}
"""


def test_forms(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    (tmp_path / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "token_adaptive_bit_amd", "csrc"), str(tmp_path / "plan.cpp"),
                    "-o", str(tmp_path / "plan")], check=True)
    lines = [f"{t} {sum(counts(e, rows, seed))} {n} {k} {key[0]} {e} {codes}"
             for key, (t, rows, seed, n, k, e, codes) in TAILS.items()]
    out = subprocess.run([str(tmp_path / "plan")], input="\n".join(lines), capture_output=True, text=True, check=True).stdout.split()
    assert [int(f) for f in out] == [key[1] for key in TAILS]


@pytest.mark.parametrize("key", sorted(TAILS), ids=str)
def test_last_round(key):
    _, form, parts = key
    all_ = tiles(key)
    left = len(all_) % UNITS
    assert len(all_) > UNITS
    assert parts == (1 if left == 0 or left > UNITS // 2 else 2 if left > UNITS // 4 else 4)
    last = all_[len(all_) - left :]
    assert any(c % 16 for c in last)
    if parts > 1:
        part = TILES[form][1] // parts
        assert any(c <= part * (parts - 1) for c in last)    # a part, or several, without tokens


def test_every_form_is_there():
    for gated in (0, 1):
        assert {key[1] for key in TAILS if key[0] == gated} == set(TILES)
        assert {key[2] for key in TAILS if key[0] == gated} == {1, 2, 4}
