"""Ragged expert products on shared tiles past one round of the units, where the tiles of the last part round are whole, halves
or quarters (tests/expert_tails.py), plain and gated, through gathered rows: against sums in float64 (exact: they stay below
2^53), every row of every expert.

Tolerances as in test_gpu_int8_linear.
"""
import pytest

torch = pytest.importorskip("torch")

from expert_tails import TAILS, counts
from test_gpu_int8_paths import BF, DEV, F32, api, weight   # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("key", sorted(TAILS), ids=lambda k: "gated%d-form%d-parts%d" % k)
def test_tails(api, key):
    gated = key[0]
    t, asked, seed, n, k, experts, codes = TAILS[key]
    print("tails", key, TAILS[key], flush=True)
    each = counts(experts, asked, seed)
    p = sum(each)
    ends = [sum(each[:e]) for e in range(experts + 1)]
    g = torch.Generator(device=DEV).manual_seed(seed)
    ws = [weight(g, experts, n, k) for _ in range(gated + 1)]
    packed = api.expert_pack_gated(ws[0][0], ws[1][0], ws[0][1], ws[1][1]) if gated else api.expert_pack(*ws[0])
    x = torch.randn(t, k, generator=g, device=DEV).to(BF)
    q, s = api.int8_quantize(x)
    offsets = torch.tensor(ends, dtype=torch.int32, device=DEV)
    rows = torch.randint(0, t, (p,), generator=g, device=DEV, dtype=torch.int32)
    at = rows.long()

    def product(w, scale):
        out = torch.empty(p, n, dtype=torch.float64, device=DEV)
        for e in range(experts):
            r = at[ends[e] : ends[e + 1]]
            out[ends[e] : ends[e + 1]] = (q[r].double() @ w[e].double().t().contiguous()) * (s[r].double()[:, None] * scale[e].double())
        return out
    refs = [product(*w) for w in ws]
    run = api.expert_gated if gated else api.expert_linear
    for out in (BF, F32):
        y = torch.full((p, n), float("nan"), dtype=out, device=DEV)
        run(packed, q if codes else x, offsets, rows, s if codes else None, y=y)
        if gated:
            gv, u = refs
            ref = gv * torch.sigmoid(gv) * u
            tol = ref.abs() * (gv.abs() + 4) * 2.0 ** -22 + 2.0 ** -125 * (gv * u).abs()
        else:
            ref = refs[0]
            tol = ref.abs() * 2.0 ** -22
        tol += ref.abs() * (2.0 ** -8 if out == BF else 0) + 1e-38
        worst = float(((y.double() - ref).abs() / tol).max())   # a row left out is NaN
        assert worst <= 1, f"{out}: {worst:.3f} of the tolerance"
