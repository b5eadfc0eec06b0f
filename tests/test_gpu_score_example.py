"""The scoring example end to end: 8-bit blocks, routed slices, norms and log probabilities
run together and say what the pieces say."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 7, 40, 130])
def test_score(t):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import score_block as S
    blocks, head, final, table = S.build(256, 640, 500, 2)
    tokens = torch.randint(0, 500, (t,), device=S.DEV, generator=torch.Generator(device=S.DEV).manual_seed(t))
    x = table[tokens]
    said = S.score(blocks, head, final, x, tokens, 0).top_ids[:, 0].to(torch.int64)
    ref = S.score(blocks, head, final, x, said, 0)
    assert (ref.rank == 1).all() and torch.equal(ref.top_ids[:, 0].to(torch.int64), said)
    assert torch.allclose(ref.logprob, ref.top_logprobs[:, 0], atol=1e-5)
    loss = [float(-S.score(blocks, head, final, x, said, b).logprob.mean()) for b in (3, 2, 1)]
    assert all(v >= 0 for v in loss)
    if t >= 40:      # over enough tokens the text scores best under the weights that wrote it, and 2 bits worst
        assert float(-ref.logprob.mean()) < loss[0] < loss[2]


def test_command():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "score_block.py"), "--tokens", "64", "--hidden", "256",
                          "--ffn", "640", "--vocab", "500"], capture_output=True, text=True, timeout=110)
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.count("perplexity") == 4
