"""Token log probabilities on the GPU against the float64 oracle.

Tolerances, with u = 2^-24: (x - m) / T is two roundings, ln s has the sum's relative error
(below 100 u: the exponential's 2 u, chains of at most 64 terms a lane, 8 joins) plus its own
rounding: 2^-16 + 2^-21 of the value is allowed.  The entropy adds q / s, a sum of the same
kind of up to ln v + the range of the row: 2^-15 + 2^-18 of the value.  Ids and ranks are exact.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
NEG = float("-inf")


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from token_adaptive_bit_amd import api
    return api


def check(api, z, targets, top, inv_t=1.0, tdt=torch.int64):
    """z: a GPU tensor of logits."""
    r = api.token_logprobs(z, torch.as_tensor(targets, dtype=tdt, device=DEV), top=top, inv_temperature=inv_t)
    lp, ent, rank, ids, best = D.token_logprobs(z.float().cpu().numpy(), targets, top, inv_t)
    for name, got, want, a, b in (("logprob", r.logprob, lp, -16, -21), ("entropy", r.entropy, ent, -15, -18),
                                  ("top", r.top_logprobs, best, -16, -21)):
        if got is None:
            assert top == 0
            continue
        got = got.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(got), np.isnan(want)), name
        assert np.array_equal(np.isneginf(got), np.isneginf(want)), name
        f = np.isfinite(want)
        assert (np.abs(got[f] - want[f]) <= 2.0 ** a + 2.0 ** b * np.abs(want[f])).all(), (name, np.abs(got[f] - want[f]).max())
    assert np.array_equal(r.rank.cpu().numpy(), rank)
    if top:
        assert np.array_equal(r.top_ids.cpu().numpy(), ids)


def logits(rng, t, v, dt, spread=2.5):
    z = rng.standard_normal((t, v)).astype(np.float32) * spread
    z[np.arange(t), rng.integers(0, v, t)] += 12 * rng.random(t)
    return torch.from_numpy(z).to(DEV, dt)


@pytest.mark.parametrize("t,v", [(1, 1), (1, 2), (3, 7), (2, 8), (5, 63), (4, 513), (1, 2048), (2, 8191), (1, 8192), (3, 8193), (5, 32768), (4, 32769), (256, 11000), (257, 11000),
                                 (1, 50021), (70, 1000), (2, 131072), (1, 262144), (2, 300000), (1, 700001), (700, 12000), (1100, 300), (1030, 9000), (1500, 5000)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_sizes(api, t, v, dt):
    print(f"logprobs t={t} v={v} {dt}", flush=True)
    rng = np.random.default_rng(t + v)
    for top in sorted({0, 1, min(v, 5), min(v, 20), min(v, 64)}):
        check(api, logits(rng, t, v, dt), rng.integers(0, v, t), top, float(rng.choice([1.0, 1.25, 0.5])))


@pytest.mark.parametrize("v", [5, 700, 9001, 70000, 270000])
def test_ties(api, v):
    """Equal logits: ranks and alternatives by ascending token, all equal among them, and +0 with -0."""
    rng = np.random.default_rng(v)
    top = min(v, 12)
    for z in (np.zeros((4, v)), np.where(rng.random((4, v)) < 0.5, 0.0, -0.0), rng.integers(-2, 3, (4, v)),
              np.full((4, v), -1e30), np.round(rng.standard_normal((4, v)) * 4) / 4):
        check(api, torch.from_numpy(z.astype(np.float32)).to(DEV), rng.integers(0, v, 4), top)
        check(api, torch.from_numpy(z.astype(np.float32)).to(DEV, BF), [0, v - 1, v // 2, v // 3], top)


@pytest.mark.parametrize("levels", [2, 40, 600, 20000])
@pytest.mark.parametrize("t,v", [(3, 90), (2, 2048), (1100, 3000), (2, 9000), (1500, 7000), (1, 140000)])
def test_long_lists(api, t, v, levels):
    """Lists of 13 to 64 over few to many different logits: from one tie for every place to none."""
    rng = np.random.default_rng(v + levels)
    z = torch.from_numpy(rng.integers(0, levels, (t, v)).astype(np.float32) * np.float32(16 / levels)).to(DEV)
    z[0, : v // 2] = NEG
    for top in (13, 33, 64):
        check(api, z, rng.integers(v // 2, v, t), top)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("v", [6, 300, 20000])
def test_masks(api, v, dt):
    """Ruled-out tokens as -infinity and as the type's lowest value; rows that leave one, few or no tokens."""
    rng = np.random.default_rng(v)
    z = logits(rng, 9, v, dt)
    low = torch.finfo(dt).min
    z[0, 1:] = NEG
    z[1, : v - 1] = NEG
    z[2] = NEG
    z[3, ::2] = NEG
    z[4] = low
    z[5, 1:] = low
    z[6, ::2] = low
    z[6, 1::2] = NEG
    z[7, : v // 2] = low
    z[8, 0] = torch.finfo(dt).max
    for targets in ([0] * 9, [v - 1] * 9, list(rng.integers(0, v, 9))):
        check(api, z, targets, min(v, 6))


def test_rows_without_a_distribution(api):
    for v in (5, 400, 30000):
        z = torch.randn(6, v, device=DEV)
        z[1, v - 1] = float("nan")
        z[2, 0] = float("inf")
        z[3, v // 2], z[3, 1] = float("inf"), float("nan")
        z[4] = float("nan")
        check(api, z, [0, v - 1, 0, 1, 2, 3], 3)
        check(api, z, [-1] * 6, 0)


@pytest.mark.parametrize("tdt", [torch.int32, torch.int64])
def test_padded_targets(api, tdt):
    z = torch.randn(6, 500, device=DEV)
    check(api, z, [-1, 500, -100, 3, 2 ** 31 - 1, 499], 2, tdt=tdt)
    if tdt == torch.int64:
        check(api, z, [2 ** 32, -2 ** 40, 2 ** 32 + 5, 0, 1, 2], 2)


@pytest.mark.parametrize("inv_t", [1e-3, 0.1, 1.0, 10.0, 1000.0])
def test_temperature(api, inv_t):
    rng = np.random.default_rng(3)
    check(api, logits(rng, 4, 3000, F32), rng.integers(0, 3000, 4), 5, inv_t)
    check(api, logits(rng, 2, 40000, F32, spread=100.0), rng.integers(0, 40000, 2), 5, inv_t)


def test_strides_and_alignment(api):
    """A vocabulary slice of a padded logits buffer, rows at odd element offsets."""
    rng = np.random.default_rng(8)
    for dt in (BF, F32):
        big = torch.randn(5, 4099, device=DEV).to(dt)
        check(api, big[:, 3:4000], rng.integers(0, 3997, 5), 7)
        check(api, big[1:2, 1:], [17], 7)


def test_ascending_and_descending(api):
    """Every logit is a new best one, and none after the first is."""
    for v in (1000, 40000):
        up = torch.arange(v, device=DEV, dtype=F32)[None] * 1e-3
        check(api, torch.cat([up, up.flip(1)]), [v - 1, v // 2], 64)


def test_long_buffer_offsets(api):
    """The last row starts past 2^32 bytes."""
    v, t = 150000, 7200
    z = torch.zeros(t, v, dtype=F32, device=DEV)
    z[t - 1] = torch.randn(v, device=DEV)
    r = api.token_logprobs(z, torch.full((t,), 5, device=DEV), top=3)
    lp, ent, rank, ids, best = D.token_logprobs(z[t - 1 :].cpu().numpy(), [5], 3, 1.0)
    assert abs(float(r.logprob[t - 1]) - lp[0]) < 1e-4 and int(r.rank[t - 1]) == rank[0]
    assert r.top_ids[t - 1].tolist() == ids[0].tolist() and r.top_ids[0].tolist() == [0, 1, 2]
    assert abs(float(r.entropy[0]) - np.log(v)) < 1e-4


def test_empty_batch_stream_and_workspace(api):
    r = api.token_logprobs(torch.empty(0, 50, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV), top=2)
    assert r.logprob.shape == (0,) and r.top_ids.shape == (0, 2)
    z, tg = torch.randn(3, 300000, device=DEV), torch.tensor([1, 2, 3], device=DEV)
    want = api.token_logprobs(z, tg, top=9)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ws = torch.empty(max(1, api.token_logprobs_workspace(3, 300000, 9)), dtype=torch.uint8, device=DEV)
        got = [api.token_logprobs(z, tg, top=9, workspace=ws) for _ in range(3)]
    s.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_graph_replays(api):
    z, tg = torch.randn(2, 270000, device=DEV), torch.tensor([7, 9], device=DEV)
    ws = torch.empty(max(1, api.token_logprobs_workspace(2, 270000, 4)), dtype=torch.uint8, device=DEV)
    api.token_logprobs(z, tg, top=4, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = api.token_logprobs(z, tg, top=4, workspace=ws)
    for i in range(4):
        z.copy_(torch.randn(2, 270000, device=DEV))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, api.token_logprobs(z, tg, top=4)))
