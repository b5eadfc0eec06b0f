"""Every form of the 8-bit integer linear and the experts' products that the plan can choose, on a shape that it chooses it
for (tests/int8_paths.py), against sums in float64 (exact: they stay below 2^53).  Sums are exact in every form, so codes
read in place, codes inside a wider buffer and float activations have to give one and the same result.

Tolerances as in test_gpu_int8_linear.
"""
import pytest

torch = pytest.importorskip("torch")

from int8_paths import FORMS, PATHS

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from token_adaptive_bit_amd import api
    return api


def weight(g, *shape):
    codes = torch.randint(-128, 128, shape, generator=g, device=DEV, dtype=torch.int8)
    scale = (torch.rand(shape[:-1], generator=g, device=DEV) + 0.5) / (74 * shape[-1] ** 0.5)
    return codes, scale


def make_offsets(g, experts, p):
    share = torch.rand(experts, generator=g, device=DEV) ** 2
    share[torch.rand(experts, generator=g, device=DEV) < 0.2] = 0
    share[-1] += 0.05
    ends = (share.cumsum(0) / share.sum() * p).round().int()
    return torch.cat([ends.new_zeros(1), ends])


def run(api, gated, t, p, n, k, experts):
    g = torch.Generator(device=DEV).manual_seed(t + n + k)
    shape = (experts, n, k) if experts else (n, k)
    ws = [weight(g, *shape) for _ in range(gated + 1)]
    pack = (api.expert_pack_gated if gated else api.expert_pack) if experts else (api.int8_pack_gated if gated else api.int8_pack)
    packed = pack(ws[0][0], ws[1][0], ws[0][1], ws[1][1]) if gated else pack(ws[0][0], ws[0][1])
    x = torch.randn(t, k, generator=g, device=DEV).to(BF)
    q, s = api.int8_quantize(x)
    rest = ()
    if experts:
        offsets = make_offsets(g, experts, p)
        rows = torch.randint(0, t, (p,), generator=g, device=DEV, dtype=torch.int32)
        rest, ends, at = (offsets, rows), offsets.tolist(), rows.long()

    def sums(w, ws_):
        if not experts:
            return (q.double() @ w.double().t().contiguous()) * (s.double()[:, None] * ws_.double())
        out = torch.zeros(p, n, dtype=torch.float64, device=DEV)
        for e in range(experts):
            if ends[e + 1] > ends[e]:
                r = at[ends[e] : ends[e + 1]]
                out[ends[e] : ends[e + 1]] = (q[r].double() @ w[e].double().t().contiguous()) * (s[r].double()[:, None] * ws_[e].double())
        return out
    refs = [sums(*w) for w in ws]
    wide = torch.full((t, k + 48), 101, dtype=torch.int8, device=DEV)
    wide[:, 16 : 16 + k] = q
    for out, act in ((BF, "silu"), (F32, "gelu_tanh")):
        def call(v, scale=None, **kw):
            kw.update({"act": act} if gated else {})
            if experts:
                return (api.expert_gated if gated else api.expert_linear)(packed, v, *rest, scale, out_dtype=out, **kw)
            return (api.int8_gated if gated else api.int8_linear)(packed, v, scale, out_dtype=out, **kw)
        y = call(q, s)
        if gated:
            gv, u = refs
            a = gv if act == "silu" else 1.5957691216057308 * (gv + 0.044715 * gv ** 3)
            ref = gv * torch.sigmoid(a) * u
            tol = ref.abs() * (a.abs() + 4) * (2.0 ** -22 if act == "silu" else 2.0 ** -21) + 2.0 ** -125 * (gv * u).abs()
        else:
            ref = refs[0]
            tol = ref.abs() * 2.0 ** -22
        tol += ref.abs() * (2.0 ** -8 if out == BF else 0) + 1e-38
        worst = float(((y.double() - ref).abs() / tol).max())
        assert worst <= 1, f"{out}: {worst:.3f} of the tolerance"
        assert torch.equal(call(wide[:, 16 : 16 + k], s), y), "codes inside a wider buffer"
        for xf in (x, x.float()):
            assert torch.equal(call(xf), y), f"{xf.dtype} activations"


@pytest.mark.parametrize("key", sorted(PATHS), ids=lambda k: "%s-gated%d-experts%d-split%d-inline%d-cut%d" % (FORMS[k[2]], k[0], k[1], *k[3:]))
def test_paths(api, key):
    t, p, n, k, experts, _ = PATHS[key]
    print("path", key, PATHS[key], flush=True)
    run(api, key[0], t, p, n, k, experts)


@pytest.mark.parametrize("t,n,k", [(12, 500, 4096), (16, 300, 3000), (5, 17, 9700)])
def test_longest_rows_quantized_within(api, t, n, k):
    """Codes of up to 48 KiB in LDS beside the waves' sums."""
    run(api, 1, t, t, n, k, 0)


def test_many_experts(api):
    run(api, 0, 300, 5000, 20, 272, 1024)
    run(api, 1, 3, 9, 20, 272, 1000)


def test_weights_past_4_gib(api):
    """Experts whose codes lie beyond 2^32 bytes, and 2^31 outputs and more."""
    experts, n, k = 36, 8192, 16384
    codes = torch.empty(experts, n, k, dtype=torch.int8, device=DEV).random_(-128, 128)
    scale = torch.rand(experts, n, device=DEV) / 1e4
    p = api.expert_pack(codes, scale)
    for each in (1, 20, 150):
        offsets = torch.arange(experts + 1, dtype=torch.int32, device=DEV) * each
        q = torch.randint(-127, 128, (experts * each, k), dtype=torch.int8, device=DEV)
        s = torch.rand(experts * each, device=DEV)
        y = api.expert_linear(p, q, offsets, None, s, out_dtype=F32)
        for e in (0, 17, experts - 1):
            r = slice(e * each, (e + 1) * each)
            ref = (q[r].double() @ codes[e].double().t().contiguous()) * (s[r].double()[:, None] * scale[e].double())
            assert bool(((y[r].double() - ref).abs() <= ref.abs() * 2.0 ** -22 + 1e-38).all())
    del codes, p, y
    t, n, k = 70001, 32768, 40
    w = torch.randint(-127, 128, (n, k), dtype=torch.int8, device=DEV)
    q, s = torch.randint(-127, 128, (t, k), dtype=torch.int8, device=DEV), torch.rand(t, device=DEV)
    y = api.int8_linear(api.int8_pack(w, torch.ones(n, device=DEV)), q, s)
    r = torch.tensor([0, 1, 65535, 65536, 65537, t - 1], device=DEV)
    ref = (q[r].double() @ w.double().t().contiguous()) * s[r].double()[:, None]
    assert bool(((y[r].double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -22)).all())


def test_offsets_that_make_no_sense(api):
    """Offsets are data: descending or far-off ones leave rows unwritten or written twice, inside y."""
    w = torch.randint(-127, 128, (300, 40, 272), dtype=torch.int8, device=DEV)
    p = api.expert_pack(w, torch.ones(300, 40, device=DEV))
    for t in (9, 2000, 9000):
        q, s = torch.ones(t, 272, dtype=torch.int8, device=DEV), torch.ones(t, device=DEV)
        whole = torch.full((t + 64, 40), 5.0, device=DEV)
        y = whole[32 : 32 + t]
        for offsets in (torch.randint(-2 ** 31, 2 ** 31 - 1, (301,), dtype=torch.int32, device=DEV),
                        torch.arange(301, 0, -1, dtype=torch.int32, device=DEV) * 31,
                        (torch.arange(301, dtype=torch.int32, device=DEV) % 2) * t):
            api.expert_linear(p, q, offsets, None, s, out_dtype=F32, y=y)
            torch.cuda.synchronize()
            assert bool((whole[:32] == 5).all()) and bool((whole[32 + t :] == 5).all())
