"""The build's look at waits that count the compiler's own loads (no GPU): it finds a load that was taken out, moved behind
the wait or left out of a peeled pass, and passes what the kernels were compiled to."""
import os

import pytest

build = pytest.importorskip("token_adaptive_bit_amd.build")

# One buffer ahead: 2 copies a pass, 4 loads a pass, 2 of them before the wait.  Awaited are the copies of the pass before;
# behind them lie 2 loads of that pass and 2 of this one.
HEAD = "_Z13direct_kernelv:\n"
WAIT = "\t;;#ASMSTART\n\ts_waitcnt vmcnt(%d) ; at most %d copies of the youngest %d\n\t;;#ASMEND\n"
COPY = "\tglobal_load_lds_dwordx4 v[4:5], off\n"
LOAD = "\tglobal_load_dwordx4 v[58:61], v2, s[48:49] offset:1024\n"
TAIL = "\ts_endpgm\n.Lfunc_end0:\n"
START = 4 * COPY + 8 * LOAD + WAIT % (10, 2, 10)


def pass_(before=2, after=2, wait=WAIT % (4, 0, 4)):
    return before * LOAD + wait + "\ts_barrier\n" + 2 * COPY + after * LOAD


def loop(body):
    return ".LBB0_1:\n" + body + "\ts_cbranch_scc1 .LBB0_1\n"


def test_a_sound_loop_passes():
    assert build._late_copies(HEAD + START + loop(pass_()) + WAIT % (0, 0, 0) + TAIL) == []
    # more loads than were counted only wait longer
    assert build._late_copies(HEAD + START + loop(pass_(3, 3)) + TAIL) == []


@pytest.mark.parametrize("body", [pass_(1, 2), pass_(2, 1), pass_(0, 0)])
def test_a_load_taken_out(body):
    (name, _, n, allowed, found), *_ = build._late_copies(HEAD + START + loop(body) + TAIL)
    assert name == "_Z13direct_kernelv" and (n, allowed) == (4, 0) and found > allowed


def test_a_load_moved_behind_the_wait():
    body = LOAD + WAIT % (4, 0, 4) + 2 * COPY + 2 * LOAD
    assert build._late_copies(HEAD + START + loop(body + "\ts_nop 0\n") + TAIL)


def test_a_last_pass_peeled_off_without_its_loads():
    assert build._late_copies(HEAD + START + loop(pass_()) + pass_(0, 0) + TAIL)
    # the pass itself may leave them out if it waits for copies alone
    assert build._late_copies(HEAD + START + loop(pass_()) + pass_(0, 0, WAIT % (0, 0, 0)) + TAIL) == []


def test_a_way_round_the_loads():
    body = "\ts_cbranch_vccz .LBB0_2\n" + 2 * LOAD + ".LBB0_2:\n" + WAIT % (4, 0, 4) + 2 * COPY + 2 * LOAD
    assert build._late_copies(HEAD + START + loop(body) + TAIL)


def test_a_kernel_whose_waits_are_gone():
    assert build._late_copies(HEAD + START.replace("; at most", "; ") + TAIL)


def test_the_kernels_as_compiled():
    path = os.path.join(build.BUILD_DIR, "int8_linear.s")
    if not os.path.exists(path):
        pytest.skip("not built here")
    with open(path) as f:
        text = f.read()
    assert build._late_copies(text) == []
    assert len(build._WAIT.findall(text)) >= 24 * 4          # 24 kernels: one wait before the loop, some in it, one behind
