"""Long top lists that are filled through a wave's LDS: 65 to 256 entries at once, after steps
that leave the list empty, in every split of a row."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
STEP = 2048                   # logits a wave reads at once


@pytest.fixture(scope="module")
def api():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from token_adaptive_bit_amd import api
    return api


@pytest.mark.parametrize("masked", [0, 1, 3])
@pytest.mark.parametrize("t,v", [(4096, 9000), (1500, 16500), (1100, 33000), (3, 140000)])
@pytest.mark.parametrize("levels", [0, 300])
def test_lists_after_empty_steps(api, t, v, masked, levels):
    print(f"lists t={t} v={v} masked={masked} levels={levels}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(v + masked + levels)
    z = torch.randn(t, v, generator=g, device=DEV)
    if levels:
        z = (z * levels / 8).round() * (8 / levels)                # many equal logits
    z[::2, : masked * STEP] = float("-inf")
    z[1::3, STEP - 5 : masked * STEP] = float("-inf")              # a few entries in the first step
    targets = torch.full((t,), v - 1, device=DEV)
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :64]
    for top in (13, 20, 64):
        r = api.token_logprobs(z, targets, top=top)
        assert torch.equal(r.top_ids.long(), order[:, :top]), top
