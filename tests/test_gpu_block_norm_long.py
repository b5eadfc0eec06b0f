"""Statistics of very long rows.

Rows of +c and -c in equal numbers have the mean 0 and the mean square c^2 exactly, whatever
the width, and their norm is +-c / sqrt(c^2 + eps).  Every addition of equal terms rounds the
same way, so that a sum in one chain drifts by up to its length times half a unit.
Tolerance, with u = 2^-24: a statistic is summed over 8 elements, 32 such vectors, up to 64
runs of those and the 1024 threads of a row (6 levels and 16 waves), so by at most 126
additions and a rounding of the square each; the square root halves it: 64 u, and 8 u for
the roundings after it.
"""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL = 72 * 2.0 ** -24


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from token_adaptive_bit_amd import api
    return api


def rows(k, dt):
    c = torch.tensor([1.1, 1.3, 0.7, 1.93, 3.3], device=DEV).to(dt)
    sign = torch.ones(k, device=DEV)
    sign[1 : k - k % 2 : 2] = -1
    if k % 2:
        sign[-1] = 0
    return c, (c[:, None] * sign.to(dt)[None]).contiguous(), sign


@pytest.mark.parametrize("k", [40000, 1 << 20, (1 << 20) + 3, 1 << 22, (1 << 24) - 8, 1 << 24])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_equal_magnitudes(api, k, kind, dt):
    print(f"long norm k={k} {kind} {dt}", flush=True)
    eps = 1e-6
    c, x, sign = rows(k, dt)
    y, h = api.block_norm(x, kind=kind, eps=eps, out_dtype=torch.float32)
    assert torch.equal(y, x)
    for i, v in enumerate(c.double().tolist()):
        want = v / math.sqrt(v * v * (k - k % 2) / k + eps)
        err = (h[i].double() - sign.double() * want).abs().max() / want
        assert float(err) <= TOL, f"row of {v}: {float(err) / TOL:.2f} of the tolerance"


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_both_norms_of_a_long_row(api, kind):
    """Ordinary values through both norms and the residual, against float64."""
    k = (1 << 21) + 5
    g = torch.Generator(device=DEV).manual_seed(4)
    x, r = (torch.randn(2, k, generator=g, device=DEV) + 0.5 for _ in range(2))

    def norm(v):
        v = v - v.mean(1, keepdim=True) if kind == "layer" else v
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)

    y, h = api.block_norm(x, r, post=torch.ones(k, device=DEV), kind=kind, residual_scale=0.9, gate_scale=1.1)
    y64 = 0.9 * r.double() + 1.1 * norm(x.double())
    h64 = norm(y64)
    assert ((y.double() - y64).abs() <= TOL * (1 + y64.abs())).all()
    assert ((h.double() - h64).abs() <= 2 * TOL * (1 + h64.abs())).all()
