"""Pins of oracle/expert_oracle.py that come from the formulas, not from the oracle itself (no GPU)."""
import numpy as np
import pytest

from oracle import expert_oracle as E


def test_quantize_by_hand():
    q, s = E.quantize(np.array([[127.0, -127.0, 0.5, 1.5, 2.5, -0.49], [0, 0, 0, 0, 0, 0]], np.float32))
    assert q.tolist() == [[127, -127, 0, 2, 2, 0], [0] * 6]                     # factor 1: ties to even
    assert s[0] == 1 and s[1] == np.float32(2.0 ** -96) / np.float32(127)
    q, s = E.quantize(np.array([[1, np.inf], [np.nan, 1], [1, 2]], np.float32))
    assert np.isnan(s[:2]).all() and (q[:2] == 0).all() and q[2].tolist() == [64, 127]   # 63.5 to even


def test_quantize_is_within_half_a_step_and_scales():
    x = np.random.default_rng(0).standard_normal((7, 300)).astype(np.float32)
    q, s = E.quantize(x)
    assert np.abs(q).max(axis=1).tolist() == [127] * 7
    assert (np.abs(q * s[:, None].astype(np.float64) - x) <= s[:, None] * (0.5 + 2.0 ** -16)).all()
    q2, s2 = E.quantize(x * 2.0 ** 9)
    assert np.array_equal(q, q2) and np.array_equal(s2, s * 2.0 ** 9)


def test_product_loop():
    rng = np.random.default_rng(1)
    xq, wq = rng.integers(-128, 128, (3, 5)).astype(np.int8), rng.integers(-128, 128, (4, 5)).astype(np.int8)
    xs, ws = rng.random(3).astype(np.float32), rng.random(4).astype(np.float32)
    y, acc = E.product(xq, xs, wq, ws)
    for i in range(3):
        for j in range(4):
            n = sum(int(a) * int(b) for a, b in zip(xq[i], wq[j]))
            assert acc[i, j] == n and y[i, j] == n * (float(xs[i]) * float(ws[j]))


def test_gate_by_its_other_forms():
    g, u = np.linspace(-5, 5, 101), np.linspace(2, 3, 101)
    assert np.allclose(E.gate(g, u, "silu"), g * u * (1 + np.tanh(g / 2)) / 2, rtol=1e-12)
    assert np.allclose(E.gate(g, u, "gelu_tanh"), u * g / 2 * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3))), rtol=1e-9)
    assert E.gate(np.array([-800.0]), np.array([1.0]), "silu")[0] == 0


def test_route_by_hand():
    inf = np.inf
    z = np.array([[0, 1, 1, -inf], [-inf] * 4, [3, -inf, -inf, -inf], [0, np.nan, 0, 0], [2, 2, 2, 2]])
    ids, w, perm, offsets, place = E.route(z, 2)
    assert ids.tolist() == [[1, 2], [-1, -1], [0, -1], [-1, -1], [0, 1]]
    assert np.allclose(w[[0, 1, 2, 4]], [[0.5, 0.5], [0, 0], [1, 0], [0.5, 0.5]]) and np.isnan(w[3]).all()
    assert offsets.tolist() == [0, 2, 4, 5, 5] and perm.tolist() == [2, 4, 0, 4, 0] + [-1] * 5
    assert place.tolist() == [[2, 4], [-1, -1], [0, -1], [-1, -1], [1, 3]]
    p = np.exp([0, 1, 1]) / np.exp([0, 1, 1]).sum()
    assert np.allclose(E.route(z, 3, normalize=False)[1][0], [p[1], p[2], p[0]])
    s = 1 / (1 + np.exp(-1.0))
    assert np.allclose(E.route(z, 3, "sigmoid", False, 2.0)[1][0], [2 * s, 2 * s, 1.0])
    assert np.allclose(E.route(z, 3, "sigmoid", True)[1].sum(1)[[0, 2, 4]], 1)


@pytest.mark.parametrize("t,e,top", [(1, 1, 1), (9, 5, 2), (40, 7, 7)])
def test_group_is_a_stable_sort(t, e, top):
    z = np.random.default_rng(t).standard_normal((t, e))
    ids, _, perm, offsets, place = E.route(z, top)
    at = np.argsort(ids.ravel(), kind="stable")
    assert np.array_equal(perm, at // top) and np.array_equal(place.ravel()[at], np.arange(t * top))
    assert np.array_equal(np.diff(offsets), np.bincount(ids.ravel(), minlength=e))


def test_combine_inverts_the_grouping():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 4))
    ids, w, perm, offsets, place = E.route(rng.standard_normal((6, 5)), 3)
    y, mags = E.combine(x[perm], w, place)
    assert np.allclose(y, x) and np.allclose(mags, np.abs(x))                   # weights of a token add up to 1
    y, _ = E.combine(x[:2], np.array([[0.5, np.nan], [1, 0]]), np.array([[0, -1], [9, -1]]), np.ones((2, 4)))
    assert np.isnan(y[0]).all() and np.array_equal(y[1], np.ones(4))
