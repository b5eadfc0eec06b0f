"""Every form of the 8-bit linear and the gated half that the plan can choose, on a shape that it
chooses it for (tests/fp8_paths.py): codes read in place from rows inside a wider buffer of NaN codes,
codes of dense rows, and float activations, against float64 and against each other.

Tolerances, relative to the sum of the products' magnitudes: for bfloat16 outputs 2^-15 (the fp8
instruction's sum stays below 2^-16 on operands of one size, and the float32 additions of up to
133 blocks, scales and joins below 2^-16), for float32 outputs 2^-24 (16 + blocks) (a block's sum
and its scale in 16 roundings, one addition a block); a rounding to bfloat16 is 2^-8 of the result.
"""
import pytest

torch = pytest.importorskip("torch")

from fp8_paths import STREAMS, TILES

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


def weight(g, n, k):
    """Codes, scales and float64 values of a weight."""
    codes = (torch.randn(n, k, generator=g, device=DEV) * 100).clamp_(-448, 448).to(F8)
    scale = (torch.rand(-(-n // 128), -(-k // 128), generator=g, device=DEV) + 0.5) / (100 * k ** 0.5)
    return codes, scale, codes.double() * scale.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]


def act(g, name):
    if name == "silu":
        return g * torch.sigmoid(g)
    return g / 2 * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)))


def run(api, t, n, k, gated, outs):
    g = torch.Generator(device=DEV).manual_seed(t + n + k)
    ws = [weight(g, n, k) for _ in range(gated + 1)]
    p = api.fp8_pack_gated(ws[0][0], ws[1][0], ws[0][1], ws[1][1]) if gated else api.fp8_pack(ws[0][0], ws[0][1])
    x = torch.randn(t, k, generator=g, device=DEV).to(BF)
    q, s = api.fp8_quantize(x)
    values = q.double() * s.double().t().repeat_interleave(128, 1)[:, :k]
    sums = [values @ w[2].t().contiguous() for w in ws]
    mags = [values.abs() @ w[2].abs().t().contiguous() for w in ws]
    wide = torch.full((t, k + 48), 0x7F, dtype=torch.uint8, device=DEV)
    wide[:, 16 : 16 + k] = q.view(torch.uint8)
    inside = wide.view(F8)[:, 16 : 16 + k]
    for out in outs:
        off = 2.0 ** -15 if out == BF else 2.0 ** -24 * (16 + -(-k // 128))
        rounding = 2.0 ** -8 if out == BF else 2.0 ** -23
        for name in ("silu", "gelu_tanh") if gated else (None,):
            def call(*a):
                return api.fp8_gated(p, *a, act=name, out_dtype=out) if gated else api.fp8_linear(p, *a, out_dtype=out)
            y = call(q, s)
            if gated:     # both activations have slopes of at most 1.13; exp and the reciprocal are good to 2^-20
                want = act(sums[0], name) * sums[1]
                tol = off * (1.13 * mags[0] * sums[1].abs() + sums[0].abs() * mags[1]) + 2.0 ** -18 * (sums[0] * sums[1]).abs()
            else:
                want, tol = sums[0], off * mags[0]
            tol = tol + rounding * want.abs() + 1e-30
            worst = float(((y.double() - want).abs() / tol).max())
            assert worst <= 1, f"{name} {out}: {worst:.3f} of the tolerance"
            assert torch.equal(call(inside, s), y), "rows inside a wider buffer"
            for xf in (x, x.float()):
                assert torch.equal(call(xf), y), f"{xf.dtype} activations"


@pytest.mark.parametrize("key", sorted(TILES), ids=lambda k: "gated%d-f32%d-tile%d-split%d" % k)
def test_tiles(api, key):
    print("tiles", key, TILES[key], flush=True)
    run(api, *TILES[key], key[0], [F32 if key[1] else BF])


@pytest.mark.parametrize("key,t", [(k, STREAMS[k][0]) for k in sorted(STREAMS)] + [(k, 1) for k in sorted(STREAMS) if k[2] == 1])
def test_streams(api, key, t):
    shape = (t, *STREAMS[key][1:])
    print("streams", key, shape, flush=True)
    run(api, *shape, key[0], [BF, F32])
