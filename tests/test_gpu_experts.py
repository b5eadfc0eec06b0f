"""The experts' route, products and combine on the GPU against the float64 oracle, and a block of experts run as a user
runs it, eagerly and from a graph.

Tolerances.  Ids, perm, offsets and place are exact.  Products as in test_gpu_int8_linear.  Weights: expf is within 2 ulp and
1 + exp adds one rounding; a sum of at most 1024 positive terms over lanes and then registers is off by less than 2^-19 of
itself, the quotient and the scale by 2^-24 each: 2^-18.  Combine: top float32 additions, 2^-24 of the terms' magnitudes
each, and one rounding to the output's type.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import expert_oracle as E
from test_gpu_int8_linear import DEV, DT, api, close, make_w, make_x, tolerance   # noqa: F401

pytestmark = pytest.mark.gpu


def check_route(api, logits, top, score="softmax", normalize=True, scale=1.0):
    r = api.expert_route(logits, top, score=score, normalize=normalize, weight_scale=scale)
    z = logits.float().cpu().numpy()
    ids, weights, perm, offsets, place = E.route(z, top, score, normalize, scale)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.perm.cpu().numpy(), perm)
    assert np.array_equal(r.place.cpu().numpy(), place)
    w = r.weights.cpu().numpy()
    assert np.array_equal(np.isnan(w), np.isnan(weights))
    bad = np.abs(w - weights) > np.abs(weights) * 2.0 ** -18 + 1e-37
    assert not bad.any()
    return r


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,e,top", [(1, 1, 1), (1, 64, 6), (17, 9, 4), (32, 64, 6), (33, 257, 9), (2, 5, 5), (64, 128, 8),
                                     (65, 128, 8), (63, 130, 2), (200, 7, 3), (1000, 256, 8), (300, 1000, 32), (257, 300, 4),
                                     (129, 64, 1), (40, 1024, 32)])
def test_route(api, t, e, top, dtype):
    rng = np.random.default_rng(t + e * 5 + top)
    z = torch.from_numpy((rng.standard_normal((t, e)) * 2).astype(np.float32)).to(DT[dtype]).to(DEV)   # bfloat16: many ties
    check_route(api, z, top)
    check_route(api, z, top, "sigmoid", False, 2.5)


@pytest.mark.parametrize("t", [5, 32, 33, 64, 90, 5000])
def test_route_masks_ties_and_bad_rows(api, t):
    rng = np.random.default_rng(t)
    z = rng.standard_normal((t, 40)).astype(np.float32)
    z[rng.random((t, 40)) < 0.5] = -np.inf
    z[:, 7] = -np.inf                                          # an expert without tokens
    z[0] = -np.inf                                             # padding
    z[1] = 0.0
    z[1, ::2] = -0.0                                           # ties of both zeros
    z[2, 3:] = -np.inf                                         # fewer than top left
    z[3, 39] = np.nan
    z[4, 0] = np.inf
    z[t // 2 + 2 :: 7] = -np.inf
    z[z < -2] = np.finfo(np.float32).min                       # allowed, and nothing of the softmax
    z = torch.from_numpy(z).to(DEV)
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            check_route(api, z, 6, score, normalize)


def test_route_long_and_strided(api):
    """Beyond a span of histograms, checked by a stable sort; rows of logits apart."""
    t, e, top = 20011, 72, 3
    big = torch.randn(t, 100, device=DEV)
    z = big[:, 11 : 11 + e]
    r = api.expert_route(z, top)
    best = z.topk(top, dim=1)
    assert torch.equal(r.ids, best.indices.int())
    flat = r.ids.flatten().long()
    order = torch.argsort(flat, stable=True)
    assert torch.equal(r.perm.long(), order // top)
    assert torch.equal(r.place.flatten()[order], torch.arange(t * top, device=DEV, dtype=torch.int32))
    assert torch.equal(r.offsets[1:].long(), torch.bincount(flat, minlength=e).cumsum(0))
    assert torch.equal(r.weights, api.expert_route(z.contiguous(), top).weights)


def test_route_of_nothing(api):
    r = api.expert_route(torch.empty(0, 30, device=DEV), 4)
    assert r.ids.shape == (0, 4) and r.perm.numel() == 0 and r.offsets.tolist() == [0] * 31


def make_groups(rng, experts, rows, skew):
    """Rows of every expert: none for some, most of them with one."""
    share = rng.random(experts) ** skew
    share[rng.random(experts) < 0.3] = 0
    share[rng.integers(experts)] += 0.1
    counts = rng.multinomial(rows, share / share.sum())
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def reference(xq, xs, parts, offsets, rows, act):
    (wq, ws) = parts[0]
    n = wq.shape[1]
    m = len(rows)
    ref, g, u = np.zeros((m, n)), np.zeros((m, n)), np.zeros((m, n))
    for e in range(len(offsets) - 1):
        at = slice(offsets[e], offsets[e + 1])
        ref[at], _ = E.product(xq[rows[at]], xs[rows[at]], wq[e], ws[e])
        if len(parts) == 2:
            g[at] = ref[at]
            u[at], _ = E.product(xq[rows[at]], xs[rows[at]], parts[1][0][e], parts[1][1][e])
    if len(parts) == 2:
        return E.gate(g, u, act), g, u
    return ref, None, None


EXPERT_SHAPES = [(1, 1, 1, 1, 1), (4, 6, 6, 100, 300), (8, 40, 17, 33, 520), (5, 100, 100, 130, 260), (3, 300, 70, 270, 1000),
                 (70, 200, 90, 48, 129), (2, 1500, 600, 160, 384), (130, 150, 40, 20, 1030), (3, 40, 9, 64, 3000)]


@pytest.mark.parametrize("experts,m,t,n,k", EXPERT_SHAPES)
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("dtype,gated", [("bf16", False), ("f32", True), ("codes", False), ("bf16", True)])
def test_products(api, experts, m, t, n, k, gather, dtype, gated):
    rng = np.random.default_rng(experts * 1000 + m + n + k)
    offsets = make_groups(rng, experts, m, 3)
    rows = rng.integers(0, t, m).astype(np.int32) if gather else np.arange(m, dtype=np.int32)
    x, xn = make_x(rng, t if gather else m, k, "f32" if dtype == "codes" else dtype)
    ws = [make_w(rng, experts, n, k) for _ in range(1 + gated)]
    xq, xs = E.quantize(xn)
    ref, g, u = reference(xq, xs, [w[1] for w in ws], offsets, rows, "silu")
    p = api.expert_pack_gated(ws[0][0], ws[1][0]) if gated else api.expert_pack(ws[0][0])
    out = torch.float32 if dtype == "f32" else torch.bfloat16
    run = api.expert_gated if gated else api.expert_linear
    scale = None
    if dtype == "codes":
        x, scale = torch.from_numpy(xq).to(DEV), torch.from_numpy(xs).to(DEV)
    y = run(p, x, torch.from_numpy(offsets).to(DEV), torch.from_numpy(rows).to(DEV) if gather else None, scale, out_dtype=out)
    close(y, ref, tolerance(ref, out, g, u, "silu"))


@pytest.mark.parametrize("m,k", [(12, 300), (200, 300), (3000, 260)])
def test_rows_behind_the_last_expert_and_bad_indices(api, m, k):
    """Rows of no expert stay as they were; an index outside x makes a row of zeros; offsets are cut to the rows there are."""
    rng = np.random.default_rng(m)
    experts, n, t = 4, 50, 30
    w, (wq, ws) = make_w(rng, experts, n, k)
    x, xn = make_x(rng, t, k, "bf16")
    xq, xs = E.quantize(xn)
    p = api.expert_pack(w)
    rows = rng.integers(0, t, m).astype(np.int32)
    offsets = np.array([0, m // 4, m // 4, m // 2, m - m // 5], np.int32)
    bad = rng.random(m) < 0.1
    given = np.where(bad, rng.choice([-1, t, 2 ** 31 - 1, -2 ** 31], m), rows).astype(np.int32)
    ref, _, _ = reference(xq, xs, [(wq, ws)], offsets, rows, None)
    ref[bad] = 0
    y = torch.full((m, n), 7.0, dtype=torch.bfloat16, device=DEV)
    api.expert_linear(p, x, torch.from_numpy(offsets).to(DEV), torch.from_numpy(given).to(DEV), y=y)
    assert bool((y[m - m // 5 :] == 7).all())
    close(y[: m - m // 5], ref[: m - m // 5], tolerance(ref[: m - m // 5], torch.bfloat16))
    # offsets past the rows and below 0 are cut
    cut = np.array([-5, m // 4, m // 4, m // 2, m + 1000], np.int32)
    ref, _, _ = reference(xq, xs, [(wq, ws)], np.clip(cut, 0, m), rows, None)
    close(api.expert_linear(p, x, torch.from_numpy(cut).to(DEV), torch.from_numpy(rows).to(DEV)), ref, tolerance(ref, torch.bfloat16))


def test_a_bad_row_spoils_only_itself(api):
    rng = np.random.default_rng(5)
    w, (wq, ws) = make_w(rng, 3, 40, 200)
    for t in (4, 300):
        x, _ = make_x(rng, t, 200, "f32")
        x[2, 100] = float("inf")
        xq, xs = E.quantize(x.cpu().numpy())
        offsets = np.array([0, 2, t - 1, t], np.int32)
        ref, _, _ = reference(xq, xs, [(wq, ws)], offsets, np.arange(t), None)
        assert np.isnan(ref[2]).all() and np.isnan(ref).sum() == 40
        close(api.expert_linear(api.expert_pack(w), x, torch.from_numpy(offsets).to(DEV)), ref, tolerance(ref, torch.float32))


@pytest.mark.parametrize("t,n,top", [(1, 1, 1), (3, 7, 2), (70, 2050, 6), (5, 5000, 32), (300, 129, 8), (1000, 64, 3)])
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("bf16", None)])
def test_combine(api, t, n, top, dtype, res):
    rng = np.random.default_rng(t + n + top)
    p = t * top
    rows = torch.from_numpy(rng.standard_normal((p, n)).astype(np.float32)).to(DT[dtype]).to(DEV)
    place = rng.integers(-1, p, (t, top)).astype(np.int32)
    weights = rng.standard_normal((t, top)).astype(np.float32)
    residual = None if res is None else torch.from_numpy(rng.standard_normal((t, n)).astype(np.float32)).to(DT[res]).to(DEV)
    ref, mags = E.combine(rows.float().cpu().numpy(), weights, place, None if residual is None else residual.float().cpu().numpy())
    y = api.expert_combine(rows, torch.from_numpy(weights).to(DEV), torch.from_numpy(place).to(DEV), residual)
    out = DT[res or dtype]
    assert y.dtype == out
    tol = mags * (top + 1) * 2.0 ** -24 + np.abs(ref) * (2.0 ** -8 if out == torch.bfloat16 else 0) + 1e-30
    close(y, ref, tol)
    if residual is not None:                                   # in place, and rows apart
        wide = torch.zeros(t, n + 9, dtype=out, device=DEV)
        wide[:, 4 : 4 + n] = residual
        inside = wide[:, 4 : 4 + n]
        assert api.expert_combine(rows, torch.from_numpy(weights).to(DEV), torch.from_numpy(place).to(DEV), inside, y=inside) is inside
        assert torch.equal(inside, y) and float(wide[:, :4].abs().max()) == 0 and float(wide[:, 4 + n :].abs().max()) == 0


def test_combine_bad_weights_and_no_rows(api):
    place = torch.tensor([[-1, 0], [-1, -1], [5, 1]], dtype=torch.int32, device=DEV)
    weights = torch.tensor([[float("nan"), 1.0], [0.0, 0.0], [3.0, 2.0]], device=DEV)
    residual = torch.ones(3, 10, device=DEV)
    y = api.expert_combine(torch.full((2, 10), 4.0, device=DEV), weights, place, residual)
    assert bool(torch.isnan(y[0]).all()) and bool((y[1] == 1).all()) and bool((y[2] == 9).all())
    y = api.expert_combine(torch.empty(0, 10, device=DEV), weights[1:2], place[1:2], residual[:1])
    assert torch.equal(y, residual[:1])


class Block:
    """The feed-forward half of a block of experts, as a user writes it."""

    def __init__(self, api, rng, experts, hidden, ffn, top):
        self.api, self.top = api, top
        (g, self.g), (u, self.u), (d, self.d) = make_w(rng, experts, ffn, hidden), make_w(rng, experts, ffn, hidden), make_w(rng, experts, hidden, ffn)
        self.gated, self.down = api.expert_pack_gated(g, u), api.expert_pack(d)

    def __call__(self, x, logits, residual):
        r = self.api.expert_route(logits, self.top)
        h = self.api.expert_gated(self.gated, x, r.offsets, r.perm)
        y = self.api.expert_linear(self.down, h, r.offsets)
        return self.api.expert_combine(y, r.weights, r.place, residual), h, y, r


@pytest.mark.parametrize("t", [1, 3, 50, 400])
def test_block_of_experts(api, t):
    rng = np.random.default_rng(t)
    experts, hidden, ffn, top = 12, 200, 130, 3
    b = Block(api, rng, experts, hidden, ffn, top)
    x, xn = make_x(rng, t, hidden, "bf16", 0, 0)
    residual = torch.randn(t, hidden, device=DEV)
    logits = torch.randn(t, experts, device=DEV)
    if t > 2:
        logits[t // 2] = float("-inf")                         # a padded token keeps its residual
    out, h, y, r = b(x, logits, residual)
    ids, weights, perm, offsets, place = E.route(logits.cpu().numpy(), top)
    used = offsets[-1]
    xq, xs = E.quantize(xn)
    ref, g, u = reference(xq, xs, [b.g, b.u], offsets, perm, "silu")
    close(h[:used], ref[:used], tolerance(ref, torch.bfloat16, g, u, "silu")[:used])
    hq, hs = E.quantize(h.float().cpu().numpy()[:used])        # each step from what the step before gave
    ref, _, _ = reference(hq, hs, [b.d], offsets, np.arange(used), None)
    close(y[:used], ref, tolerance(ref, torch.bfloat16))
    ref, mags = E.combine(y.float().cpu().numpy()[:used], r.weights.cpu().numpy(), place, residual.cpu().numpy())
    close(out, ref, mags * (top + 1) * 2.0 ** -24 + 1e-30)
    if t > 2:
        assert torch.equal(out[t // 2], residual[t // 2])


@pytest.mark.parametrize("t", [2, 130])
def test_block_captured_and_replayed(api, t):
    rng = np.random.default_rng(t + 1)
    b = Block(api, rng, 10, 256, 192, 2)
    x, logits, residual = torch.randn(t, 256, device=DEV, dtype=torch.bfloat16), torch.randn(t, 10, device=DEV), torch.randn(t, 256, device=DEV)
    b(x, logits, residual)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = b(x, logits, residual)[0]
    for i in range(4):
        x.normal_()
        logits.normal_()
        if i == 2:
            logits[0] = float("-inf")
        want = b(x, logits, residual)[0]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want)


def test_on_another_stream(api):
    rng = np.random.default_rng(2)
    b = Block(api, rng, 6, 256, 192, 2)
    x, logits, residual = torch.randn(40, 256, device=DEV), torch.randn(40, 6, device=DEV), torch.randn(40, 256, device=DEV)
    want = b(x, logits, residual)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = b(x, logits, residual)[0]
    s.synchronize()
    assert torch.equal(got, want)


def test_two_streams_at_once(api):
    rng = np.random.default_rng(3)
    b = Block(api, rng, 9, 300, 200, 3)
    args = [(torch.randn(t, 300, device=DEV, dtype=torch.bfloat16), torch.randn(t, 9, device=DEV), torch.randn(t, 300, device=DEV))
            for t in (700, 33)]
    want = [b(*a)[0] for a in args]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(10):
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                got.append(b(*a)[0])
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])


def test_two_graphs_share_a_workspace(api):
    """Replayed one after the other: nothing that a call leaves in its workspace is read by the next."""
    rng = np.random.default_rng(4)
    w, _ = make_w(rng, 5, 190, 330)
    p = api.expert_pack(w)
    wide, _ = make_w(rng, 1, 70, 16000)
    q = api.int8_pack(wide[0])
    x, logits = torch.randn(90, 330, device=DEV, dtype=torch.bfloat16), torch.randn(90, 5, device=DEV)
    z = torch.randn(100, 16000, device=DEV)
    need = max(api.int8_workspace(p, 90, rows=180), api.int8_workspace(q, 100, torch.float32), api.expert_route_workspace(90, 5))
    workspace = torch.empty(need, dtype=torch.uint8, device=DEV)
    a, b = torch.empty(180, 190, device=DEV), torch.empty(100, 70, device=DEV)

    def first():
        r = api.expert_route(logits, 2, workspace=workspace)
        return api.expert_linear(p, x, r.offsets, r.perm, y=a, workspace=workspace)

    def second():
        return api.int8_linear(q, z, y=b, workspace=workspace)

    first(), second()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, f in zip(graphs, (first, second)):
        with torch.cuda.graph(g):
            f()
    for i in range(3):
        x.normal_()
        logits.normal_()
        z.normal_()
        r = api.expert_route(logits, 2)
        want = api.expert_linear(p, x, r.offsets, r.perm, out_dtype=torch.float32), api.int8_linear(q, z)
        a.zero_()
        b.zero_()
        for k in (0, 1, 0) if i % 2 else (1, 0, 1):
            graphs[k].replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
