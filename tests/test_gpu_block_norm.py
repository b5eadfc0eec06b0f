"""Norms around a block on the GPU against the float64 oracle.

Tolerances, with u = 2^-24: y is three float32 operations on z, and z's own error is that
of a norm; a norm's error is that of its sums (trees over at most 32 terms a lane and 10
levels: below 24 u, halved by the square root) plus a few roundings, 32 u of the value in
all; subtracting the mean adds 4 u of the largest input times 1 / std.  Twice that is
allowed.  bfloat16 outputs add one rounding (2^-9, 2^-8 allowed).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from token_adaptive_bit_amd import api
    return api


def dev(a, dt=F32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV, dt)


def back(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(api, t, k, xd=F32, rd=F32, hd=F32, kind="rms", post=True, gate="none", residual=True, bias=False,
          quantized=False, offset=0.0, seed=0, a=0.9, b=1.1, eps=1e-6):
    rng = np.random.default_rng(seed + t * 131 + k)
    x = dev(rng.standard_normal((t, k)) * 3 + offset, xd)
    r = dev(rng.standard_normal((t, k)) * 2 + offset, rd) if residual else None
    pre, pst = (1 + 0.2 * rng.standard_normal(k)).astype(np.float32), (1 + 0.2 * rng.standard_normal(k)).astype(np.float32)
    pb, qb = (rng.standard_normal((2, k)) if bias else (None, None))
    gn = {"none": None, "channel": rng.random(k), "token": rng.random(t), "full": rng.random((t, k))}[gate]
    gt = None if gn is None else dev(gn, xd if gate == "full" else F32)
    out = api.block_norm(x, r, pre=dev(pre), post=dev(pst) if post else None, gate=gt, residual_scale=a, gate_scale=b,
                         eps=eps, kind=kind, pre_bias=dev(pb) if bias else None,
                         post_bias=dev(qb) if bias and post else None, quantized=quantized,
                         out_dtype=None if quantized else hd)
    g64 = None if gn is None else back(gt)[:, None] if gate == "token" else back(gt)
    y64, h64, rstd, mags = D.block_norm(back(x), None if r is None else back(r), pre, pst if post else None, g64, a, b, eps, kind,
                                        None if pb is None else dev(pb).cpu().numpy(), None if qb is None or not post else dev(qb).cpu().numpy())
    torch.cuda.synchronize()
    y = out[0]
    assert y.dtype == (rd if residual else xd)
    wmax = np.abs(pst).max() if post else 1.0
    _, rx = D.norm(back(x), None, None, kind, eps)
    mean_term = (4 * U * np.abs(back(x)).max(1, keepdims=True) * rx * wmax * b) if kind == "layer" and post else 0.0
    ytol32 = 2 * (40 * U * mags + mean_term + (8 * U * np.abs(qb).max() * b if bias and post else 0))
    ytol = ytol32 + (np.abs(y64) * 2.0 ** -8 if y.dtype == BF else 0) + 1e-30
    worst = (np.abs(back(y) - y64) / ytol).max()
    assert worst <= 1, f"y: {worst:.2f} of the tolerance"
    row = np.abs(y64).max(1, keepdims=True)
    htol = 2 * (32 * U * np.abs(h64) + (ytol32.max(1, keepdims=True) + 4 * U * row) * rstd * np.abs(pre).max()
                + (8 * U * np.abs(pb).max() if bias else 0)) + 1e-30
    if quantized:
        q, s = out[1], out[2]
        assert q.dtype == F8 and s.shape == (-(-k // 128), t)
        sv = np.repeat(back(s).T, 128, axis=1)[:, :k]
        amax = np.abs(np.pad(h64, ((0, 0), (0, -k % 128)))).reshape(t, -1, 128).max(2)
        assert (np.abs(back(s).T - amax / 448) <= htol.max() / 448 + amax * 4 * U / 448).all()
        codes = q.contiguous().view(torch.uint8).cpu().numpy()
        err = np.abs(D.e4m3_values()[codes] * sv - h64)       # half a step: 2^-4 of the value, 2^-10 of the scale below it
        assert (err <= np.abs(h64) * 2.0 ** -4 * 1.001 + sv * 2.0 ** -10 + 2 * htol).all()
        plain = api.block_norm(x, r, pre=dev(pre), post=dev(pst) if post else None, gate=gt, residual_scale=a, gate_scale=b,
                               eps=eps, kind=kind, pre_bias=dev(pb) if bias else None,
                               post_bias=dev(qb) if bias and post else None, out_dtype=F32)[1]
        q2, s2 = api.fp8_quantize(plain)                      # the same h, quantized apart: the same codes
        assert torch.equal(s, s2) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
    else:
        h = out[1]
        worst = (np.abs(back(h) - h64) / (htol + (np.abs(h64) * 2.0 ** -8 if h.dtype == BF else 0))).max()
        assert worst <= 1, f"h: {worst:.2f} of the tolerance"


WIDTHS = [1, 2, 7, 8, 64, 127, 128, 129, 250, 256, 257, 500, 512, 513, 1000, 1531, 2048, 2056, 4096, 4100, 5120, 8192, 8200, 13824, 16384,
          17000, 18944, 25000, 32768, 33000]


@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_widths(api, k, kind):
    print(f"block norm k={k} {kind}", flush=True)
    check(api, 5, k, kind=kind, bias=kind == "layer")
    check(api, 3, k, xd=BF, rd=BF, kind=kind, gate="channel", quantized=True)


@pytest.mark.parametrize("xd,rd,hd", [(BF, BF, BF), (BF, F32, BF), (F32, BF, F32), (BF, F32, F32), (F32, F32, BF)])
@pytest.mark.parametrize("k", [77, 1024, 5120, 17000])
def test_types(api, xd, rd, hd, k):
    check(api, 4, k, xd=xd, rd=rd, hd=hd, gate="full")


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("k", [130, 2100, 16500])
def test_parts(api, gate, post, residual, k):
    check(api, 6, k, xd=BF, rd=BF, gate=gate, post=post, residual=residual, kind="layer", bias=True)


@pytest.mark.parametrize("t", [0, 1, 2, 3, 4, 5, 63, 1000])
@pytest.mark.parametrize("k", [40, 96, 200, 640, 1500])
def test_rows(api, t, k):
    if t == 0:
        y, h = api.block_norm(torch.empty(0, k, device=DEV), None)
        assert y.shape == h.shape == (0, k)
    else:
        check(api, t, k)
        check(api, t, k, quantized=True)


@pytest.mark.parametrize("t,k", [(5000, 100), (5001, 200), (4200, 500), (3000, 700), (2000, 1500), (1203, 2100), (700, 6000), (300, 18944)])
@pytest.mark.parametrize("quantized", [False, True])
def test_many_rows(api, t, k, quantized):
    """Enough rows for the form that keeps fewer registers."""
    check(api, t, k, xd=BF, rd=BF, hd=BF, kind="layer", gate="channel", bias=True, quantized=quantized)


def test_large_mean(api):
    """Layer norm where the mean is 1000 times the deviation: the variance is taken about it."""
    for k in (300, 4096, 20000):
        check(api, 3, k, kind="layer", offset=3000.0, post=False)


def test_missing_weights_are_ones(api):
    x = torch.randn(4, 300, device=DEV)
    y, h = api.block_norm(x)
    _, h1 = api.block_norm(x, pre=torch.ones(300, device=DEV))
    assert torch.equal(y, x) and torch.equal(h, h1)


def test_zero_and_non_finite_rows(api):
    """A row of zeros norms to zeros (to the bias for a layer norm); a NaN or infinity stays in its row."""
    for k in (40, 1000, 17000):
        x = torch.randn(5, k, device=DEV)
        x[1] = 0
        x[2, k // 2] = float("nan")
        x[3, k - 1] = float("inf")
        clean = api.block_norm(torch.nan_to_num(x, nan=0.0, posinf=0.0))[1]
        y, h = api.block_norm(x)
        assert (h[1] == 0).all() and torch.isnan(h[2]).all() and torch.isnan(h[3, k - 1])
        assert torch.equal(h[[0, 1, 4]], clean[[0, 1, 4]])
        _, q, s = api.block_norm(x, quantized=True)
        assert (q[1].float() == 0).all() and torch.isfinite(s[:, 1]).all() and torch.isnan(s[:, 2]).all()
        bias = torch.randn(k, device=DEV)
        assert torch.equal(api.block_norm(x[1:2], kind="layer", pre_bias=bias)[1][0], bias)


@pytest.mark.parametrize("k", [90, 1536, 9000, 20000])
def test_in_place_and_strides(api, k):
    """y over residual, inputs and outputs as column ranges of wider buffers at odd offsets."""
    for dt in (BF, F32):
        x, r = (torch.randn(7, k, device=DEV).to(dt) for _ in range(2))
        w = torch.rand(k, device=DEV) + 0.5
        y, h = api.block_norm(x, r, pre=w, post=w, residual_scale=0.7)
        r2 = r.clone()
        y2, h2 = api.block_norm(x, r2, pre=w, post=w, residual_scale=0.7, y=r2)
        assert y2 is r2 and torch.equal(y, y2) and torch.equal(h, h2)
        big = torch.zeros(4, 7, k + 37, device=DEV, dtype=dt)
        big[0, :, 3 : 3 + k], big[1, :, 5 : 5 + k] = x, r
        y3, h3 = api.block_norm(big[0, :, 3 : 3 + k], big[1, :, 5 : 5 + k], pre=w, post=w, residual_scale=0.7,
                                y=big[2, :, 1 : 1 + k], h=big[3, :, 7 : 7 + k])
        assert torch.equal(y, y3) and torch.equal(h, h3)
        assert not big[2, :, 0].any() and not big[2, :, 1 + k :].any() and not big[3, :, 7 + k :].any()


def test_feeds_the_linear(api):
    """The quantized output is the linear's operand: the same result as from h in float32."""
    for t in (1, 16, 100):
        x, r = torch.randn(t, 640, device=DEV).bfloat16(), torch.randn(t, 640, device=DEV).bfloat16()
        p = api.fp8_pack(torch.randn(96, 640, device=DEV))
        _, q, s = api.block_norm(x, r, quantized=True)
        _, h = api.block_norm(x, r, out_dtype=F32)
        assert torch.equal(api.fp8_linear(p, q, s), api.fp8_linear(p, h, out_dtype=BF))
