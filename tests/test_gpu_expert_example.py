"""The scoring example on blocks of experts: quantization, route, experts' products, combine, norms and log probabilities run
together and say what the same stack of plain products says."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 7, 40, 300])
def test_score(t):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import score_block as S
    blocks, head, final, table = S.build_experts(256, 640, 500, 2, 12)
    tokens = torch.randint(0, 500, (t,), device=S.DEV, generator=torch.Generator(device=S.DEV).manual_seed(t))
    x = table[tokens]
    said = S.score_experts(blocks, head, final, x, tokens, 4).top_ids[:, 0].to(torch.int64)
    ref = S.score_experts(blocks, head, final, x, said, 4)
    assert (ref.rank == 1).all() and torch.equal(ref.top_ids[:, 0].to(torch.int64), said)
    assert torch.allclose(ref.logprob, ref.top_logprobs[:, 0], atol=1e-5)
    again = S.score_experts(blocks, head, final, x, said, 4)
    assert torch.equal(again.logprob, ref.logprob)      # no atomics: a second run is the first bit for bit
    for n in (1, 2, 12):
        r = S.score_experts(blocks, head, final, x, said, n)
        assert torch.isfinite(r.logprob).all() and (r.logprob <= 0).all()


def test_score_in_a_graph():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import score_block as S
    blocks, head, final, table = S.build_experts(256, 640, 500, 2, 12)
    tokens = torch.arange(70, device=S.DEV)
    x = table[tokens].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        S.score_experts(blocks, head, final, x, tokens, 2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = S.score_experts(blocks, head, final, x, tokens, 2)
    for first in (0, 100, 400):
        x.copy_(table[first:first + 70])
        graph.replay()
        torch.cuda.synchronize()
        want = S.score_experts(blocks, head, final, x, tokens, 2)
        assert torch.equal(r.logprob, want.logprob) and torch.equal(r.top_ids, want.top_ids)


def test_command():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "score_block.py"), "--tokens", "64", "--hidden", "256",
                          "--ffn", "640", "--vocab", "500", "--experts", "6"], capture_output=True, text=True, timeout=110)
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.count("experts a token: perplexity") == 3
