"""The last digits of log probabilities and entropies, where one token is all but certain.

Tolerances, with u = 2^-24.  Every term is held about a reference within a factor of 2^1.5 of
the largest one, so a confident row's s lies between 0.5 and 3 and ln s and the target's exponent
are numbers of order 1.  The log probability's error is that of s (a lane adds one sum of 8 terms
for every 512 logits of its part: at most 12 of them here with one part a row, 10 with four, 4 with
more; each addition rounds by u s at most and by a third of that on the mean, in either
direction, so sqrt(12) u for the chain, 3 u for a vector's terms and exponentials and 8 joins),
of ln and of two products: below 8 u = 2^-21.  The entropy adds q / s, whose terms are the
entropy's own: below 8 u (1 + H).  With terms of up to 2^16 in s both sums are off by several times that.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from token_adaptive_bit_amd import api
    return api


@pytest.mark.parametrize("boost", [9.0, 10.5, 12.0, 16.0, 30.0])
@pytest.mark.parametrize("t,v", [(4096, 6000), (1100, 20000), (64, 20000), (64, 50021), (8, 128000)])
def test_confident_rows(api, t, v, boost):
    print(f"confident rows t={t} v={v} boost={boost}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(v + int(boost))
    z = torch.randn(t, v, generator=g, device=DEV)
    targets = torch.randint(0, v, (t,), generator=g, device=DEV)
    z[torch.arange(t, device=DEV), targets] = boost + torch.rand(t, generator=g, device=DEV)
    r = api.token_logprobs(z, targets, top=1)
    assert torch.equal(r.top_ids[:, 0].long(), targets) and (r.rank == 1).all()
    for lo in range(0, t, 512):
        rows = slice(lo, min(lo + 512, t))
        logp = torch.log_softmax(z[rows].double(), 1)
        want = logp.gather(1, targets[rows, None])[:, 0]
        entropy = -(logp.exp() * logp).sum(1)
        err = (r.logprob[rows].double() - want).abs() / (2.0 ** -21 * (1 + want.abs()))
        assert float(err.max()) <= 1, f"log probability: {float(err.max()):.2f} of the tolerance"
        assert torch.equal(r.top_logprobs[rows, 0], r.logprob[rows])
        err = (r.entropy[rows].double() - entropy).abs() / (2.0 ** -21 * (1 + entropy))
        assert float(err.max()) <= 1, f"entropy: {float(err.max()):.2f} of the tolerance"


def test_growing_rows(api):
    """Logits that outgrow the reference in every step, in one part and in many, at several temperatures."""
    for t, v in ((4096, 8000), (3, 131072)):
        z = (torch.arange(v, device=DEV) * (40.0 / v)).repeat(t, 1)
        z[:, ::2] -= 3.0
        targets = torch.full((t,), v - 1, device=DEV)
        for inv_t in (0.25, 1.0, 8.0):
            r = api.token_logprobs(z, targets, top=2, inv_temperature=inv_t)
            logp = torch.log_softmax(z[0].double() * inv_t, 0)
            entropy = -(logp.exp() * logp).sum()
            assert ((r.logprob.double() - logp[-1]).abs() <= 2.0 ** -20 * (1 - logp[-1])).all()
            assert ((r.entropy.double() - entropy).abs() <= 2.0 ** -20 * (1 + entropy)).all()
