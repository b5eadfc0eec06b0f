"""8-bit integer quantization, linear and gated half on the GPU against the float64 oracle.

Tolerances.  Codes, scales and sums are exact.  A finished sum is rounded to float32, multiplied by the product of two
scales, itself rounded: three roundings of 2^-24, 2^-22 allowed.  A gate's exponent moves by the rounding of its argument:
silu(g) by at most (|g| + 4) 2^-22 of itself, gelu by (|a| + 4) 2^-21 with a = 2 sqrt(2 / pi) (g + 0.044715 g^3) (four more
roundings); where exp overflows the reciprocal's flush leaves 2^-125 |g u|.  The output's rounding is 2^-24 for float32
(inside the above) and 2^-8 for bfloat16.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import expert_oracle as E

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
OUT = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from token_adaptive_bit_amd import api
    return api


def make_x(rng, t, k, dtype, lo=-3, hi=3):
    x = rng.standard_normal((t, k)) * np.exp2(rng.integers(lo, hi + 1, (t, 1)))
    if k > 4:
        x[:, rng.integers(0, k)] *= 20
    x = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
    return x.to(DEV), x.float().numpy()


def make_w(rng, *shape):
    w = (rng.standard_normal(shape) / np.sqrt(shape[-1]) * np.exp2(rng.integers(-2, 3, shape[:-1] + (1,)))).astype(np.float32)
    return torch.from_numpy(w).to(DEV), E.quantize(w)


def tolerance(ref, out_dtype, g=None, u=None, act=None):
    tol = np.abs(ref) * (OUT[out_dtype] + 2.0 ** -22)
    if g is not None:
        a = np.abs(g) if act == "silu" else np.abs(1.5957691216057308 * (g + 0.044715 * g ** 3))
        tol = np.abs(ref) * (OUT[out_dtype] + (a + 4) * (2.0 ** -22 if act == "silu" else 2.0 ** -21)) + 2.0 ** -125 * np.abs(g * u)
    return tol + 1e-38


def close(y, ref, tol):
    y = y.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(y), np.isnan(ref))
    worst = np.nanmax(np.abs(y - ref) / tol) if ref.size and not np.isnan(ref).all() else 0.0
    assert worst <= 1.0, f"error is {worst:.3f} of the tolerance"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,k", [(1, 1), (1, 128), (3, 7), (5, 129), (17, 1000), (64, 2048), (66, 2049), (130, 3584), (2, 8200),
                                 (70, 8193), (2, 18944), (3, 40001)])
def test_quantize_is_exact(api, t, k, dtype):
    rng = np.random.default_rng(t * 7919 + k)
    x, _ = make_x(rng, t, k, dtype, -30, 30)
    if t > 2:
        x[1] = 0                                             # a token of zeros
        x[2, : k // 2] = 1e-36
    q, s = api.int8_quantize(x)
    codes, scale = E.quantize(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), scale) and np.array_equal(q.cpu().numpy(), codes)


def test_quantize_ties_edges_and_bad_rows(api):
    """Every half step with a row maximum of 127 (factor 1), the smallest and largest maxima, infinities and NaN."""
    half = np.arange(-254, 255, dtype=np.float32) / 2
    x = np.zeros((6, 600), np.float32)
    x[0, : len(half)] = half
    x[1, 5], x[2, 7], x[3, 599] = np.finfo(np.float32).max, np.inf, np.nan
    x[4, 0], x[5, 3] = 2.0 ** -96, -(2.0 ** -126)
    q, s = api.int8_quantize(torch.from_numpy(x).to(DEV))
    codes, scale = E.quantize(x)
    assert np.array_equal(s.cpu().numpy(), scale, equal_nan=True) and np.array_equal(q.cpu().numpy(), codes)


def test_quantize_strided_rows(api):
    big = torch.randn(9, 700, device=DEV)
    x = big[:, 3:303]
    out = torch.full((9, 320), 77, dtype=torch.int8, device=DEV)
    q, s = api.int8_quantize(x, q=out[:, :300])
    codes, scale = E.quantize(x.cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), scale) and np.array_equal(q.cpu().numpy(), codes)
    assert bool((out[:, 300:] == 77).all())


@pytest.mark.parametrize("experts,n,k,gated", [(1, 1, 1, False), (1, 17, 129, False), (3, 40, 300, False), (2, 50, 260, True)])
@pytest.mark.parametrize("source", ["f32", "bf16", "codes"])
def test_pack_blob(api, experts, n, k, gated, source):
    """Every code and scale of the blob at the place the format gives it."""
    rng = np.random.default_rng(n + k)
    ws = [torch.from_numpy(rng.standard_normal((experts, n, k)).astype(np.float32)).to(DT.get(source, torch.float32)) for _ in range(1 + gated)]
    qs = [E.quantize(w.float().numpy()) for w in ws]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    scales = [None, None]
    if source == "codes":
        scales = [torch.from_numpy(s).to(DEV) for _, s in qs]
        ws = [torch.from_numpy(c) for c, _ in qs]
    ws = [w.to(DEV) for w in ws]
    d = api.int8_describe(n, k, gated, experts)
    fill = torch.full((int(d.total_bytes),), 0xAB, dtype=torch.uint8, device=DEV)
    p = api.expert_pack_gated(ws[0], ws[1], scales[0], scales[1], status=status, out=fill) if gated else \
        api.expert_pack(ws[0], scales[0], status=status, out=fill)
    blob = p.blob.cpu().numpy()
    assert int(status) == 0 and (p.experts, p.n, p.k, p.gated) == (experts, n, k, gated)
    parts = 1 + gated
    want = np.zeros((experts, d.row_blocks, d.k_blocks, 2, 4, 16, 16), np.int8)   # e, rb, kb, h, c, r, byte
    want_s = np.zeros((experts, d.row_blocks, 16), np.float32)
    for part, (codes, s) in enumerate(qs):
        pad = np.zeros((experts, d.row_blocks // parts * 16, d.k_blocks * 128), np.int8)
        pad[:, :n, :k] = codes
        want[:, part::parts] = pad.reshape(experts, -1, 16, d.k_blocks, 2, 4, 16).transpose(0, 1, 3, 4, 5, 2, 6)
        pad = np.zeros((experts, d.row_blocks // parts * 16), np.float32)
        pad[:, :n] = s
        want_s[:, part::parts] = pad.reshape(experts, -1, 16)
    assert np.array_equal(blob[: d.scales_offset].view(np.int8), want.reshape(-1))
    assert np.array_equal(blob[d.scales_offset : d.scales_offset + want_s.size * 4].view(np.float32), want_s.reshape(-1))


def test_pack_reports_non_finite_weights(api):
    w = torch.randn(20, 40, device=DEV)
    for bad, codes in ((float("nan"), False), (float("inf"), False), (float("nan"), True)):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        if codes:
            s = torch.ones(20, device=DEV)
            s[7] = bad
            api.int8_pack(torch.ones(20, 40, dtype=torch.int8, device=DEV), s, status=status)
        else:
            v = w.clone()
            v[3, 39] = bad
            api.int8_pack(v, status=status)
        assert int(status) == 1


SHAPES = [(1, 1, 1), (1, 16, 128), (1, 5000, 260), (2, 17, 16), (3, 100, 1000), (5, 33, 5000), (16, 130, 129), (4, 48, 20000),
          (17, 1, 130), (33, 100, 300), (64, 256, 128), (65, 300, 1000), (100, 70, 3000), (130, 1000, 257), (257, 530, 384),
          (300, 513, 1030), (1, 40, 8200), (1030, 260, 256), (700, 2050, 520)]


@pytest.mark.parametrize("t,n,k", SHAPES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("codes", "f32")])
def test_linear(api, t, n, k, dtype, out):
    rng = np.random.default_rng(t * 31 + n * 7 + k)
    x, xn = make_x(rng, t, k, "f32" if dtype == "codes" else dtype)
    w, (wq, ws) = make_w(rng, n, k)
    p = api.int8_pack(w)
    xq, xs = E.quantize(xn)
    if dtype == "codes":
        y = api.int8_linear(p, torch.from_numpy(xq).to(DEV), torch.from_numpy(xs).to(DEV), out_dtype=DT[out])
    else:
        y = api.int8_linear(p, x, out_dtype=DT[out])
    ref, _ = E.product(xq, xs, wq, ws)
    assert y.dtype == DT[out] and y.shape == (t, n)
    close(y, ref, tolerance(ref, DT[out]))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (1, 100, 1000), (7, 17, 129), (16, 130, 2000), (17, 40, 300), (65, 100, 260),
                                   (200, 300, 500), (520, 130, 257)])
def test_gated(api, t, n, k, act):
    rng = np.random.default_rng(t + n * 3 + k)
    x, xn = make_x(rng, t, k, "bf16")
    (wg, (gq, gs)), (wu, (uq, us)) = make_w(rng, n, k), make_w(rng, n, k)
    p = api.int8_pack_gated(wg, wu)
    xq, xs = E.quantize(xn)
    (g, _), (u, _) = E.product(xq, xs, gq, gs), E.product(xq, xs, uq, us)
    ref = E.gate(g, u, act)
    for out in (torch.bfloat16, torch.float32):
        close(api.int8_gated(p, x, act=act, out_dtype=out), ref, tolerance(ref, out, g, u, act))


@pytest.mark.parametrize("t", [3, 40, 300])
def test_sums_are_exact_at_full_range(api, t):
    """Codes of -128 and 127 over a row as long as the format takes: the sum reaches 2^31 - 2^14 and is not rounded on the way."""
    k, n = (1 << 17) - 1, 20
    w = torch.full((n, k), -128, dtype=torch.int8, device=DEV)
    w[1::2] = 127
    x = torch.full((t, k), -128, dtype=torch.int8, device=DEV)
    x[1::2] = 127
    p = api.int8_pack(w, torch.ones(n, device=DEV))
    y = api.int8_linear(p, x, torch.ones(t, device=DEV), out_dtype=torch.float32).cpu().numpy()
    xn, wn = np.where(np.arange(t) % 2, 127, -128), np.where(np.arange(n) % 2, 127, -128)
    assert np.array_equal(y, (xn[:, None] * wn[None] * k).astype(np.float32))


@pytest.mark.parametrize("t", [2, 30, 200])
def test_bad_tokens_spoil_only_themselves(api, t):
    rng = np.random.default_rng(t)
    x, _ = make_x(rng, t, 300, "bf16")
    w, (wq, ws) = make_w(rng, 70, 300)
    x[1, 299], x[0, 3] = float("nan"), float("-inf")
    xq, xs = E.quantize(x.float().cpu().numpy())
    ref, _ = E.product(xq, xs, wq, ws)
    assert np.isnan(ref[:2]).all() and not np.isnan(ref[2:]).any()
    close(api.int8_linear(api.int8_pack(w), x), ref, tolerance(ref, torch.bfloat16))


@pytest.mark.parametrize("t,k", [(3, 304), (3, 300), (50, 304), (50, 300), (200, 304)])
def test_rows_apart(api, t, k):
    """Float rows and codes apart from each other, at odd places where that is allowed."""
    rng = np.random.default_rng(k + t)
    w, (wq, ws) = make_w(rng, 90, k)
    p = api.int8_pack(w)
    big = torch.randn(t, k + 33, device=DEV, dtype=torch.bfloat16)
    x = big[:, 5 : 5 + k]
    xq, xs = E.quantize(x.float().cpu().numpy())
    ref, _ = E.product(xq, xs, wq, ws)
    close(api.int8_linear(p, x), ref, tolerance(ref, torch.bfloat16))
    lead = 16 if k % 16 == 0 else 3
    codes = torch.full((t, k + 48), 99, dtype=torch.int8, device=DEV)
    codes[:, lead : lead + k] = torch.from_numpy(xq).to(DEV)
    close(api.int8_linear(p, codes[:, lead : lead + k], torch.from_numpy(xs).to(DEV)), ref, tolerance(ref, torch.bfloat16))


def test_given_buffers_empty_batches_and_repeats(api):
    w = torch.randn(100, 500, device=DEV)
    p = api.int8_pack(w)
    assert api.int8_linear(p, torch.empty(0, 500, device=DEV)).shape == (0, 100)
    x = torch.randn(90, 500, device=DEV)
    y = torch.empty(90, 100, device=DEV)
    ws = torch.empty(api.int8_workspace(p, 90, torch.float32), dtype=torch.uint8, device=DEV)
    assert api.int8_linear(p, x, y=y, workspace=ws) is y
    for _ in range(3):
        assert torch.equal(api.int8_linear(p, x), y)
