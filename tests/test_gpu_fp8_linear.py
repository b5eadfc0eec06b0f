"""8-bit quantization, linear and gated half on the GPU against the float64 oracle.

Tolerances.  Codes and scales are exact.  A product's error has three parts: the matrix
instruction's own sum over a block (measured at up to 3.8e-5 of the block's sum of
magnitudes; 2^-14 = 6.1e-5 is allowed), the float32 sum over blocks (below 2^-16 of the sum
of magnitudes for the block counts here), and one rounding of the output (2^-9 for
bfloat16; 2^-8 is allowed so that a value on the edge may land on either side).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


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


def make_w(rng, n, k):
    return (rng.standard_normal((n, k)) / np.sqrt(k)).astype(np.float32)


def codes_of(q):
    return q.contiguous().view(torch.uint8).cpu().numpy()


def close(y, ref, mags, out, extra=0.0):
    y = y.float().cpu().numpy().astype(np.float64)
    tol = mags * (2.0 ** -14 + 2.0 ** -16) + np.abs(ref) * (2.0 ** -8 if out == "bf16" else 2.0 ** -22) + extra + 1e-30
    worst = (np.abs(y - ref) / tol).max() if ref.size else 0.0
    assert worst <= 1.0, f"error is {worst:.3f} of the tolerance"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,k", [(1, 1), (1, 128), (3, 7), (5, 129), (17, 1000), (64, 256), (130, 3584), (2, 18944)])
def test_quantize_is_exact(api, t, k, dtype):
    rng = np.random.default_rng(t * 7919 + k)
    x, xn = make_x(rng, t, k, dtype, -30, 30)
    if t > 2:
        x[1], xn[1] = 0, 0                                   # a token of zeros
        x[2, : k // 2], xn[2, : k // 2] = 1e-36, np.float32(1e-36) if dtype == "f32" else x[2, :1].float().cpu().numpy()
        xn = x.float().cpu().numpy()
    q, s = api.fp8_quantize(x)
    codes, scale = D.quantize(xn)
    torch.cuda.synchronize()
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(codes_of(q), codes)


def test_quantize_ties_and_edges(api):
    """Every e4m3 value and every midpoint between two, with a block maximum of 448 (factor 1)."""
    v = D.e4m3_values()[:127]
    x = np.concatenate([v, (v[:-1] + v[1:]) / 2, [448.0] * 3]).astype(np.float32)
    x = np.concatenate([x, -x])
    x = np.concatenate([x, np.zeros(-len(x) % 128, np.float32)]).reshape(-1, 128)
    x[:, 0] = 448.0
    q, s = api.fp8_quantize(torch.from_numpy(x).to(DEV))
    codes, scale = D.quantize(x)
    assert np.array_equal(s.cpu().numpy(), scale) and np.array_equal(codes_of(q), codes)


def test_quantize_strided_rows(api):
    big = torch.randn(9, 700, device=DEV)
    x = big[:, 3:303]                                        # rows at odd element offsets, stride 700
    out = torch.zeros(9, 320, dtype=torch.uint8, device=DEV).view(F8)
    q, s = api.fp8_quantize(x, q=out[:, :300])
    codes, scale = D.quantize(x.cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), scale) and np.array_equal(codes_of(q), codes)
    assert int(out.view(torch.uint8)[:, 300:].max()) == 0    # nothing past k is written


@pytest.mark.parametrize("n,k,gated", [(1, 1, False), (16, 128, False), (17, 129, False), (300, 700, False),
                                       (128, 256, True), (50, 300, True)])
@pytest.mark.parametrize("source", ["f32", "bf16", "codes"])
def test_pack_blob(api, n, k, gated, source):
    """Every code and scale of the blob at the place the format gives it."""
    rng = np.random.default_rng(n + k)
    parts = [make_w(rng, n, k) for _ in range(2 if gated else 1)]
    if source == "bf16":
        parts = [torch.from_numpy(w).bfloat16().float().numpy() for w in parts]
    qs = [D.quantize_weight(w) for w in parts]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if source == "codes":
        ws = [torch.from_numpy(c).to(DEV).view(F8) for c, _ in qs]
        ss = [torch.from_numpy(s).to(DEV) for _, s in qs]
    else:
        ws, ss = [torch.from_numpy(w).to(DEV, DT[source]) for w in parts], [None, None]
    fill = torch.full((int(api.fp8_describe(n, k, gated).total_bytes),), 0xAB, dtype=torch.uint8, device=DEV)
    p = api.fp8_pack_gated(ws[0], ws[1], ss[0], ss[1], status=status, out=fill) if gated else \
        api.fp8_pack(ws[0], ss[0], status=status, out=fill)
    blob, d = p.blob.cpu().numpy(), p.desc
    assert int(status) == 0
    want = np.zeros((d.row_blocks, d.k_blocks, 2, 4, 16, 16), np.uint8)   # rb, kb, h, c, r, e
    for part, (codes, _) in enumerate(qs):
        pad = np.zeros((d.row_blocks // len(qs) * 16, d.k_blocks * 128), np.uint8)
        pad[:n, :k] = codes
        want[part::len(qs)] = pad.reshape(-1, 16, d.k_blocks, 2, 4, 16).transpose(0, 2, 3, 4, 1, 5)
    assert np.array_equal(blob[: d.scales_offset], want.reshape(-1))
    scales = np.stack([s for _, s in qs])
    got = blob[d.scales_offset : d.scales_offset + scales.size * 4].view(np.float32).reshape(scales.shape)
    assert np.array_equal(got, scales)


def test_pack_reports_non_finite(api):
    for bad in (float("nan"), float("inf")):
        w = torch.zeros(40, 200, device=DEV)
        w[33, 150] = bad
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        api.fp8_pack(w, status=status)
        assert int(status) == 1
    for code in (0x7F, 0xFF):
        for at in ((0, 0), (39, 199), (20, 63), (7, 190)):
            q = torch.zeros(40, 200, dtype=torch.uint8, device=DEV)
            q[:] = 0x7E                                      # the largest value is no NaN
            ok, status = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
            api.fp8_pack(q.view(F8), torch.ones(1, 2, device=DEV), status=ok)
            q[at] = code
            api.fp8_pack(q.view(F8), torch.ones(1, 2, device=DEV), status=status)
            assert int(ok) == 0 and int(status) == 1


SHAPES = [  # t, n, k: one token to several tiles, every remainder that a tile can have
    (1, 1, 1), (1, 17, 128), (1, 512, 2176), (2, 130, 256), (15, 100, 300), (16, 256, 1024), (17, 48, 130),
    (31, 33, 512), (33, 200, 1100), (63, 512, 256), (64, 272, 384), (65, 30, 200), (100, 300, 129), (129, 520, 640),
    (256, 256, 256), (257, 255, 128), (300, 1000, 777), (513, 700, 400), (1500, 3000, 300), (4096, 3584, 256),
    (70, 100, 9000), (600, 520, 4000), (12, 64, 2048), (13, 64, 2048), (3, 4200, 4096), (3, 4200, 4097), (2000, 2050, 130), (1, 256, 18944), (16, 64, 18944),
    (2090, 4090, 300), (700, 6150, 200), (700, 1500, 8000), (570, 3590, 7900),
    (32, 4100, 3000), (32, 4100, 3200), (64, 512, 4096), (64, 500, 4100), (48, 530, 6150)]


@pytest.mark.parametrize("t,n,k", SHAPES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
def test_linear(api, t, n, k, dtype, out):
    print(f"fp8 linear t={t} n={n} k={k} {dtype}", flush=True)
    rng = np.random.default_rng(t * 31 + n * 7 + k)
    x, xn = make_x(rng, t, k, dtype)
    w = make_w(rng, n, k)
    p = api.fp8_pack(torch.from_numpy(w).to(DEV))
    y = api.fp8_linear(p, x, out_dtype=DT[out])
    ref, mags = D.linear(D.values_x(*D.quantize(xn)), D.values_w(*D.quantize_weight(w)))
    close(y, ref, mags, out)
    again = api.fp8_linear(p, x, out_dtype=DT[out])
    assert torch.equal(y, again)                             # the same sums in the same order


@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (1, 100, 300), (7, 144, 640), (16, 128, 128), (20, 70, 513), (64, 33, 256),
                                   (65, 128, 300), (200, 300, 256), (300, 129, 1000), (3, 64, 18944),
                                   (1030, 2100, 256), (130, 40, 6000), (520, 1000, 700), (700, 4090, 400), (1100, 4090, 300),
                                   (2040, 4000, 300)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
def test_gated(api, t, n, k, act, dtype, out):
    print(f"fp8 gated t={t} n={n} k={k} {act} {dtype}", flush=True)
    rng = np.random.default_rng(t * 13 + n + k)
    x, xn = make_x(rng, t, k, dtype, -2, 2)
    wg, wu = make_w(rng, n, k), make_w(rng, n, k)
    p = api.fp8_pack_gated(torch.from_numpy(wg).to(DEV), torch.from_numpy(wu).to(DEV))
    y = api.fp8_gated(p, x, act=act, out_dtype=DT[out])
    xv = D.values_x(*D.quantize(xn))
    g, gm = D.linear(xv, D.values_w(*D.quantize_weight(wg)))
    u, um = D.linear(xv, D.values_w(*D.quantize_weight(wu)))
    # both activations have slopes of at most 1.13; exp and the reciprocal are good to 2^-20
    extra = (2.0 ** -14 + 2.0 ** -16) * (1.13 * gm * np.abs(u) + np.abs(g) * um) + 2.0 ** -18 * np.abs(g * u)
    close(y, D.act(g, act) * u, np.zeros_like(gm), out, extra)


@pytest.mark.parametrize("t,n,k", [(1, 64, 16), (4, 100, 256), (16, 40, 144), (40, 256, 400), (70, 300, 272), (260, 128, 1040)])
def test_linear_on_codes(api, t, n, k):
    """Codes given by the caller (dense, and rows inside a wider buffer whose other bytes are
    NaN codes) give what the call on the activations gives."""
    rng = np.random.default_rng(t + n + k)
    x, _ = make_x(rng, t, k, "bf16")
    p = api.fp8_pack(torch.from_numpy(make_w(rng, n, k)).to(DEV))
    want = api.fp8_linear(p, x)
    q, s = api.fp8_quantize(x)
    assert torch.equal(api.fp8_linear(p, q, s), want)
    wide = torch.full((t, k + 48), 0x7F, dtype=torch.uint8, device=DEV)
    wide[:, 16 : 16 + k] = q.view(torch.uint8)
    assert torch.equal(api.fp8_linear(p, wide.view(F8)[:, 16 : 16 + k], s), want)


@pytest.mark.parametrize("t,n,k", [(1, 64, 7), (4, 100, 300), (16, 40, 129), (40, 256, 1001), (70, 300, 777), (260, 128, 1033)])
@pytest.mark.parametrize("gated", [False, True])
def test_codes_of_odd_rows(api, t, n, k, gated):
    """Codes with k % 16 != 0, dense and as odd rows of an odd buffer of NaN codes, and the
    codes of a norm of that width."""
    rng = np.random.default_rng(t + n + k)
    x, _ = make_x(rng, t, k, "bf16")
    w = [torch.from_numpy(make_w(rng, n, k)).to(DEV) for _ in range(2)]
    p = api.fp8_pack_gated(*w) if gated else api.fp8_pack(w[0])
    call = api.fp8_gated if gated else api.fp8_linear
    q, s = api.fp8_quantize(x)
    want = call(p, x)
    assert torch.equal(call(p, q, s), want)
    wide = torch.full((t, k + 33), 0x7F, dtype=torch.uint8, device=DEV)
    wide[:, 5 : 5 + k] = q.view(torch.uint8)
    assert torch.equal(call(p, wide.view(F8)[:, 5 : 5 + k], s), want)
    _, hq, hs = api.block_norm(x, quantized=True)
    ref = [D.linear(D.values_x(codes_of(hq), hs.cpu().numpy()), D.values_w(*D.quantize_weight(v.cpu().numpy()))) for v in w]
    (g, gm), (u, um) = ref
    if gated:
        extra = (2.0 ** -14 + 2.0 ** -16) * (1.13 * gm * np.abs(u) + np.abs(g) * um) + 2.0 ** -18 * np.abs(g * u)
        close(call(p, hq, hs), D.act(g, "silu") * u, np.zeros_like(gm), "bf16", extra)
    else:
        close(call(p, hq, hs), g, gm, "bf16")


def test_copies_of_a_weight(api):
    """A weight copied with all it holds stands alone: the first one may go."""
    import copy
    rng = np.random.default_rng(3)
    x, _ = make_x(rng, 5, 200, "bf16")
    p = api.fp8_pack(torch.from_numpy(make_w(rng, 70, 200)).to(DEV))
    want = api.fp8_linear(p, x)
    other = copy.deepcopy(p)
    p.blob.zero_()
    del p
    assert torch.equal(api.fp8_linear(other, x), want)


def test_strided_and_unaligned_activations(api):
    rng = np.random.default_rng(5)
    p = api.fp8_pack(torch.from_numpy(make_w(rng, 100, 300)).to(DEV))
    for t in (1, 16, 40, 70):
        for dt in (torch.bfloat16, torch.float32):
            big = torch.randn(t, 911, device=DEV).to(dt)
            x = big[:, 5:305]
            assert torch.equal(api.fp8_linear(p, x), api.fp8_linear(p, x.contiguous()))


@pytest.mark.parametrize("t", [1, 5, 16, 40, 64, 80, 300])
def test_tokens_do_not_touch_each_other(api, t):
    """A token with a NaN or an infinity spoils its own row only; zero tokens give zeros."""
    rng = np.random.default_rng(t)
    x, _ = make_x(rng, t, 300, "bf16")
    p = api.fp8_pack(torch.from_numpy(make_w(rng, 70, 300)).to(DEV))
    clean = api.fp8_linear(p, x)
    bad = x.clone()
    bad[0, 17] = float("nan")
    if t > 2:
        bad[t - 1, 299] = float("-inf")
        bad[1] = 0
    y = api.fp8_linear(p, bad)
    assert torch.isnan(y[0]).all()
    if t > 2:
        assert torch.isnan(y[t - 1]).all() and (y[1] == 0).all()
        assert torch.equal(y[2 : t - 1], clean[2 : t - 1])


def test_empty_batch(api):
    p = api.fp8_pack(torch.randn(20, 40, device=DEV))
    assert api.fp8_linear(p, torch.empty(0, 40, device=DEV)).shape == (0, 20)
    q, s = api.fp8_quantize(torch.empty(0, 40, device=DEV))
    assert q.shape == (0, 40) and s.shape == (1, 0)


def test_other_stream_and_given_buffers(api):
    """The call runs on the current stream, in the caller's buffers, twice in a row on a
    shared workspace."""
    rng = np.random.default_rng(9)
    w = make_w(rng, 256, 512)
    s = torch.cuda.Stream()
    p = api.fp8_pack(torch.from_numpy(w).to(DEV))
    xs = [make_x(rng, t, 512, "bf16") for t in (40, 3, 130)]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        ws = torch.empty(max(api.fp8_linear_workspace(p, t) for t in (40, 3, 130)), dtype=torch.uint8, device=DEV)
        ys = [api.fp8_linear(p, x, workspace=ws, y=torch.empty(len(x), 256, dtype=torch.bfloat16, device=DEV)) for x, _ in xs]
    s.synchronize()
    for (x, xn), y in zip(xs, ys):
        ref, mags = D.linear(D.values_x(*D.quantize(xn)), D.values_w(*D.quantize_weight(w)))
        close(y, ref, mags, "bf16")


@pytest.mark.parametrize("t", [1, 30, 100])
def test_graph_replays(api, t):
    """Captured once, replayed on new inputs in place, against the eager call."""
    rng = np.random.default_rng(t)
    p = api.fp8_pack(torch.from_numpy(make_w(rng, 200, 640)).to(DEV))
    x, _ = make_x(rng, t, 640, "bf16")
    ws = torch.empty(max(1, api.fp8_linear_workspace(p, t)), dtype=torch.uint8, device=DEV)
    y = torch.empty(t, 200, dtype=torch.bfloat16, device=DEV)
    api.fp8_linear(p, x, y=y, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.fp8_linear(p, x, y=y, workspace=ws)
    for i in range(4):
        x.copy_(make_x(np.random.default_rng(100 + i), t, 640, "bf16")[0])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, api.fp8_linear(p, x.clone()))
