"""Launches of the 8-bit integer linear (no GPU): csrc/int8_plan.h compiled by itself.  Every plan's grid holds the tiles it
has to, stays below the 2^32 threads that a launch takes (more are cut without an error), and what would not is refused."""
import ctypes
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
// t p n k gated experts codes -> does the launch hold it, threads along x, workgroups along y
int main() {
  int t, p, n, k, gated, experts, codes;
  while (std::scanf("%d %d %d %d %d %d %d", &t, &p, &n, &k, &gated, &experts, &codes) == 7) {
    const int groups = (n + 15) / 16, kb = (k + 127) / 128;
    const mbq::Int8Plan q = mbq::plan_int8(t, p, experts, groups, gated + 1, kb, codes);
    const mbq::Int8Grid g = mbq::grid_int8(q, p, experts, groups, gated + 1);
    const mbq::Int8Cost& c = mbq::kInt8Costs[int(q.form)];
    std::printf("%d %lld %lld %d %d %d %d %d\n", int(mbq::holds_int8(g)), (long long)g.x * g.threads, (long long)g.y, g.threads, int(q.form),
                q.chunks, c.rows, c.tokens);
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def grid(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("int8_launch")
    (d / "grid.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I",
                    os.path.join(ROOT, "token_adaptive_bit_amd", "csrc"), str(d / "grid.cpp"), "-o", str(d / "grid")], check=True)

    def run(cases):
        res = subprocess.run([str(d / "grid")], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True)
        assert res.returncode == 0, (res.returncode, res.stderr[-500:])
        return [tuple(map(int, line.split())) for line in res.stdout.splitlines()]
    return run


def shapes(count, most, seed):
    """Shapes that mbq_int8_describe and mbq_int8_linear accept, of at most `most` outputs."""
    rng = random.Random(seed)

    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    out = []
    while len(out) < count:
        experts, gated = rng.choice([0, 0, 1, log_int(1, 1024), 1024]), rng.randint(0, 1)
        n, k = log_int(1, 1 << 24), rng.choice([1, 128, log_int(1, (1 << 17) - 1)])
        if (n + 15) // 16 * (gated + 1) * ((k + 127) // 128) * 2048 * max(experts, 1) >= 1 << 36:
            continue
        t = log_int(1, 1 << 21)
        p = min(1 << 24, most // n) if rng.random() < 0.5 else log_int(1, 1 << 24)
        if not experts:
            t = p = min(p, 1 << 21)
        if p < 1 or p * n > most:
            continue
        out.append((t, p, n, k, gated, experts, rng.randint(0, 1)))
    return out


def test_up_to_2_37_outputs_are_held(grid):
    cases = shapes(20000, 1 << 37, 1)
    for case, (holds, threads, y, *_) in zip(cases, grid(cases)):
        assert holds and threads < 1 << 32 and y < 1 << 16, case


def test_no_launch_is_cut(grid):
    """Beyond them a launch holds all of its threads or is refused."""
    cases = shapes(20000, (1 << 38) - 1, 2) + [(3, 1021584, 269070, 128, 1, 997, 1), (11260, 10618375, 25887, 1175, 1, 1024, 1)]
    got = grid(cases)
    assert all(holds == (threads < 1 << 32 and y < 1 << 16) for holds, threads, y, *_ in got)
    assert [g[0] for g in got[-2:]] == [0, 0]


def test_grids_hold_every_tile(grid):
    """However the rows are spread over the experts."""
    rng = random.Random(3)
    cases = shapes(3000, 1 << 37, 4)
    for case, (_, threads, y, each, form, chunks, rows, tokens) in zip(cases, grid(cases)):
        t, p, n, k, gated, experts, codes = case
        if experts:
            cuts = sorted(rng.randint(0, p) for _ in range(experts - 1))
            counts = [b - a for a, b in zip([0] + cuts, cuts + [p])]
        else:
            counts = [t]
        tiles_t = sum(-(-c // tokens) for c in counts)
        tiles_n = (n + 15) // 16 if form < 3 else -(-((n + 15) // 16 * (gated + 1) * 16) // rows)
        if form < 3:
            assert threads // each == tiles_n and y >= tiles_t
        else:
            assert y == 1 and threads // each >= tiles_n * tiles_t * chunks + (512 if form >= 9 else 0)


def test_too_many_outputs_are_refused():
    """Before anything is launched: the pointers are not ones, and there need be no GPU."""
    pytest.importorskip("torch")
    from token_adaptive_bit_amd import _lib
    at = 0x7F0000000000
    for t, p, n, k, experts in ((3, 1021584, 269070, 128, 997), (11260, 10618375, 25887, 1175, 1024)):
        d = _lib.int8_describe(n, k, True, experts)
        a = _lib.MbqInt8Args(t, p, _lib.MBQ_INT8, _lib.MBQ_BF16, 0, 0, at, at, at, at, at, at, 1 << 40, (k + 15) // 16 * 16)
        with pytest.raises(_lib.MbqError, match="SHAPE|shape"):
            _lib.check(_lib.LIB.mbq_int8_linear(ctypes.byref(d), at, ctypes.byref(a), None), "mbq_int8_linear")
