"""The sum of a block's products, for both output types, on codes and scales that are given.

bfloat16 outputs take the fp8 instruction's own sum: in groups of 8 inputs products are cut
toward zero to a multiple of 2^(E - 13), E the group's largest sum of exponents (codes below
2^-6 count as 2^-6), so it is off by at most 7 * 2^-13 of the magnitudes, such codes counted as
2^-6.  Tolerances, relative to the sum of the products' magnitudes: 2^-20 for everything that is
done in float32 (the groups' or the bfloat16 instructions' additions, at most 9 roundings of
2^-24, the scale's product, one addition for each of the at most 4 blocks and the join), and
2^-8 of the result for a rounding to bfloat16.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from token_adaptive_bit_amd import api
    return api


def values(g, rows, k, kind):
    def integers(lo, hi):
        return torch.randint(lo, hi, (rows, k), generator=g, device=DEV).double()

    if kind == "subnormal":
        return integers(-7, 8) * 2.0 ** -9
    lo, hi = {"level": (6, 8), "wide": (-9, 9), "towering": (-6, 0)}[kind]
    v = torch.exp2(integers(lo, hi)) * (1 + integers(0, 8) / 8) * (integers(0, 2) * 2 - 1)
    return v.clamp(-448, 448).to(F8).double()


def operands(g, t, n, k, kind):
    """Codes' values x [t, k], w [n, k]."""
    if kind == "cut":               # one large product in eight, of alternating sign, and seven that lie just below its unit
        x, w = torch.full((t, k), 1.875 * 2.0 ** -6, device=DEV).double(), torch.full((n, k), 1.875 * 2.0 ** 7, device=DEV).double()
        x[:, ::8], w[:, ::8], w[:, ::16] = 256, -256, 256
        return x, w
    x, w = values(g, t, k, "wide" if kind == "mixed" else kind), values(g, n, k, "subnormal" if kind == "mixed" else kind)
    if kind == "towering":          # two pairs a block that cancel
        for b in range(0, k, 128):
            at = b + torch.randperm(128, generator=g, device=DEV)[:4]
            x[:, at] = torch.randint(6, 15, (t, 1), generator=g, device=DEV).double() * 32
            w[:, at[:2]] = torch.randint(6, 15, (n, 1), generator=g, device=DEV).double() * 32
            w[:, at[2:]] = -w[:, at[:2]]
    return x, w


def instruction(x, w):
    """The fp8 instruction's sums by the rule above, block by block: [t, n, blocks]."""
    t, k = x.shape
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6)))[:, None] + torch.floor(torch.log2(w.abs().clamp_min(2.0 ** -6)))[None]
    p = x[:, None] * w[None]
    e = torch.where(p == 0, -99.0, e).view(t, len(w), k // 8, 8).amax(3, keepdim=True)
    unit = torch.exp2(e - 13)
    cut = (p.view(t, len(w), k // 8, 8) / unit).trunc() * unit
    return cut.sum(3).view(t, len(w), k // 128, 16).sum(3)


@pytest.mark.parametrize("kind", ["level", "wide", "subnormal", "mixed", "towering", "cut"])
@pytest.mark.parametrize("t,n,k", [(1, 16, 128), (16, 40, 512), (40, 64, 256), (70, 48, 384), (300, 33, 512)])
def test_block_sums(api, kind, t, n, k):
    print(f"block sums t={t} n={n} k={k} {kind}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(t + n + k)
    x, w = operands(g, t, n, k, kind)
    kb = k // 128
    xs = torch.rand(kb, t, generator=g, device=DEV) + 0.5
    ws = torch.rand(1, kb, generator=g, device=DEV) + 0.5
    p = api.fp8_pack(w.to(F8), ws)
    scale = xs.double().t()[:, None] * ws.double()[None]                       # [t, 1, kb]
    blocks = [slice(128 * b, 128 * b + 128) for b in range(kb)]

    def product(a, b):
        return sum(a[:, s] @ b[:, s].t().contiguous() * scale[:, :, i] for i, s in enumerate(blocks))

    want, mags = product(x, w), product(x.abs(), w.abs())
    floored = product(x.abs().clamp_min(2.0 ** -6), w.abs().clamp_min(2.0 ** -6))
    y = api.fp8_linear(p, x.to(F8), xs, out_dtype=BF).double()
    bound = 7 * 2.0 ** -13 * floored + 2.0 ** -20 * mags + 2.0 ** -8 * want.abs()
    assert ((y - want).abs() <= bound).all(), f"{float(((y - want).abs() / bound).max()):.3f} of the bound"
    model = (instruction(x, w) * scale).sum(2)
    tol = 2.0 ** -20 * mags + 2.0 ** -8 * model.abs()
    assert ((y - model).abs() <= tol).all(), f"{float(((y - model).abs() / tol).max()):.3f} of the tolerance"
    if kind == "cut":               # all of what is not cancelled is cut
        assert (y == 0).all() and (want > 7 * 2.0 ** -14 * mags).all()
    y = api.fp8_linear(p, x.to(F8), xs, out_dtype=F32).double()
    tol = 2.0 ** -20 * mags
    assert ((y - want).abs() <= tol).all(), f"float32: {float(((y - want).abs() / tol).max()):.3f} of the tolerance"
