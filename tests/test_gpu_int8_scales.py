"""The integer linear and the experts' products where the product of a token's and an output's scale leaves float32: the
definition multiplies three numbers, so a sum of 0 gives 0 and small products keep their digits, whatever the scales.

Tolerances.  A sum is rounded to float32 and multiplied by two scales: three roundings of 2^-24, 2^-22 allowed, and a result
below 2^-126 is rounded to a multiple of 2^-149 (bfloat16: 2^-134), within 1e-38; outputs in bfloat16 add 2^-8.  A value past
float32's range is infinite.  A gate as in test_gpu_int8_linear: silu(g) moves by at most (|g| + 4) 2^-22 of itself, and where
exp overflows the reciprocal's flush leaves 2^-125 |g u|.
"""
import pytest

torch = pytest.importorskip("torch")

from int8_paths import FORMS, PATHS
from test_gpu_int8_paths import BF, DEV, F32, api, make_offsets   # noqa: F401

pytestmark = pytest.mark.gpu
# scale of a token and of an output; products of the sums below 2^31 with a pair are in float32's range where the test says so
TOKEN = (2.0 ** -70 * 1.25, 2.0 ** -7, 2.0 ** 60, 1.5 * 2.0 ** -90)
OUTPUT = (1.75 * 2.0 ** -72, 2.0 ** -14, 2.0 ** 90, 2.0 ** -30)


def scales(values, count):
    return torch.tensor(values, device=DEV).repeat(-(-count // len(values)))[:count]


@pytest.mark.parametrize("key", sorted(PATHS), ids=lambda k: "%s-gated%d-experts%d-split%d-inline%d-cut%d" % (FORMS[k[2]], k[0], k[1], *k[3:]))
def test_scales(api, key):
    gated = key[0]
    t, p, n, k, experts, given = PATHS[key]
    print("scales", key, PATHS[key], flush=True)
    g = torch.Generator(device=DEV).manual_seed(n + k)
    shape = (experts, n, k) if experts else (n, k)

    def weight(values):
        w = torch.randint(-128, 128, shape, generator=g, device=DEV, dtype=torch.int8)
        w[..., 2::8, :] = 0                                  # outputs of the largest scale whose sums are 0
        return w, scales(values, n).expand(shape[:-1]).contiguous()
    # a gate is float32: those past its range are not asked for
    ws = [weight((2.0 ** -14, 2.0 ** -14, 2.0 ** 90, 2.0 ** 40) if gated else OUTPUT)] + ([weight(OUTPUT)] if gated else [])
    if gated:                                                # the largest scales meet sums of 0 only
        ws[0][0][..., 2::4, :] = 0
        ws[0][0][..., 3::4, :] = 0
        ws[1][0][..., 2::4, :] = 0
    pack = (api.expert_pack_gated if gated else api.expert_pack) if experts else (api.int8_pack_gated if gated else api.int8_pack)
    packed = pack(ws[0][0], ws[1][0], ws[0][1], ws[1][1]) if gated else pack(ws[0][0], ws[0][1])
    x = (torch.randn(t, k, generator=g, device=DEV) * (scales(TOKEN, t) * 32.0)[:, None]).to(BF)
    x[4::5] = 0
    q, s = api.int8_quantize(x)
    if given:                                                # rows of zeros under every scale
        s = torch.where(s < 1e-30, scales(TOKEN, t), s)
    rest = ()
    if experts:
        offsets = make_offsets(g, experts, p)
        rows = torch.randint(0, t, (p,), generator=g, device=DEV, dtype=torch.int32)
        rest, ends, at = (offsets, rows), offsets.tolist(), rows.long()

    def product(w, scale):
        if not experts:
            return (q.double() @ w.double().t().contiguous()) * s.double()[:, None] * scale.double()
        out = torch.zeros(p, n, dtype=torch.float64, device=DEV)
        for e in range(experts):
            if ends[e + 1] > ends[e]:
                r = at[ends[e] : ends[e + 1]]
                out[ends[e] : ends[e + 1]] = (q[r].double() @ w[e].double().t().contiguous()) * s[r].double()[:, None] * scale[e].double()
        return out
    refs = [product(*w) for w in ws]
    for out in (BF, F32):
        kw = {"act": "silu", "out_dtype": out} if gated else {"out_dtype": out}
        run = (api.expert_gated if gated else api.expert_linear) if experts else (api.int8_gated if gated else api.int8_linear)
        y = (run(packed, q, *rest, s, **kw) if given else run(packed, x, *rest, **kw)).double()
        if gated:
            gv, u = refs
            ref = gv * torch.sigmoid(gv) * u
            tol = ref.abs() * (gv.abs() + 4) * 2.0 ** -22 + 2.0 ** -125 * (gv * u).abs()
        else:
            ref = refs[0]
            tol = ref.abs() * 2.0 ** -22
        tol += ref.abs() * (2.0 ** -8 if out == BF else 0) + 1e-38
        big = ref.abs() >= 2.0 ** 128 * (1 + 2.0 ** -20)
        assert not torch.isnan(y).any()
        if not gated:
            assert torch.equal(y[big], torch.sign(ref[big]) * float("inf"))
            assert not torch.isinf(y[ref.abs() < 2.0 ** 127]).any()
        fine = ref.abs() < 2.0 ** 127
        worst = float(((y - ref).abs() / tol)[fine].max())
        assert worst <= 1, f"{out}: {worst:.3f} of the tolerance"
