"""The scoring example on blocks of experts against the same stack in float64: every step from the weights that the stack holds
(read back from their blobs) and from what the step before gave, so that a wrong expert, a wrong weight, a wrong place or a
shared half left out shows in the step's own tolerance.

Tolerances.  Products, gates and the combine as in test_gpu_int8_linear and test_gpu_experts, norms as in
test_gpu_block_norm (64 u with u = 2^-24, and 2^-8 for bfloat16), log probabilities as in test_gpu_token_logprobs.  Ids, places, ranks, codes and
scales are exact.
"""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import dense_oracle as D
from oracle import expert_oracle as E
from test_gpu_experts import reference
from test_gpu_int8_linear import api, close, tolerance   # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
STEPS = ("block_norm", "int8_quantize", "int8_linear", "expert_route", "int8_gated", "expert_gated", "expert_linear",
         "expert_combine", "token_logprobs")


def back(t):
    return t.float().cpu().numpy()


def weights(p):
    """[(codes [experts, n, k], scale [experts, n])] of a blob's one or two weights."""
    d, blob = p.desc, p.blob.cpu().numpy()
    tiles = blob[: d.scales_offset].view(np.int8).reshape(d.experts, d.row_blocks, d.k_blocks, 2, 4, 16, 16)   # ..., half, c, r, byte
    codes = tiles.transpose(0, 1, 5, 2, 3, 4, 6).reshape(d.experts, d.row_blocks, 16, d.k_blocks * 128)
    scale = blob[d.scales_offset : d.scales_offset + 64 * d.experts * d.row_blocks].view(np.float32).reshape(d.experts, d.row_blocks, 16)
    parts = 1 + d.gated
    return [(codes[:, i::parts].reshape(d.experts, -1, d.k_blocks * 128)[:, : d.n, : d.k], scale[:, i::parts].reshape(d.experts, -1)[:, : d.n])
            for i in range(parts)]


def product(xq, xs, weight):
    (codes, scale), = weights(weight)
    return E.product(xq, xs, codes[0], scale[0])[0]


def check_norm(h, y, pre):
    """h of the float64 sum y."""
    ref = y / np.sqrt((y * y).mean(1, keepdims=True) + 1e-6) * pre.cpu().numpy().astype(np.float64)
    close(h, ref, np.abs(ref) * (2.0 ** -8 + 64 * 2.0 ** -24) + 1e-38)


@pytest.mark.parametrize("t,experts,top", [(1, 6, 2), (7, 12, 4), (40, 12, 1), (300, 12, 3)])
def test_stack(api, monkeypatch, t, experts, top):
    import score_block as S
    blocks, head, final, table = S.build_experts(192, 320, 500, 2, experts)
    g = torch.Generator(device=S.DEV).manual_seed(t)
    tokens = torch.randint(0, 500, (t,), device=S.DEV, generator=g)
    x = table[torch.randint(0, 500, (t,), device=S.DEV, generator=g)]
    made = {name: [] for name in STEPS}

    def keep(name):
        call = getattr(api, name)

        def kept(*args, **kwargs):
            made[name].append(call(*args, **kwargs))
            return made[name][-1]
        monkeypatch.setattr(S.api, name, kept)
    for name in STEPS:
        keep(name)
    result = S.score_experts(blocks, head, final, x, tokens, top)
    monkeypatch.undo()

    def take(name):
        return made[name].pop(0)
    residual, out = back(x).astype(np.float64), None
    for b in blocks:
        y, h = take("block_norm")
        whole = residual if out is None else residual + back(out)
        close(y, whole, np.abs(whole) * (2.0 ** -8 if out is not None else 2.0 ** -24) + 1e-38)
        check_norm(h, whole, b.pre)
        residual = back(y).astype(np.float64)
        q, s = take("int8_quantize")
        xq, xs = E.quantize(back(h))
        assert np.array_equal(q.cpu().numpy(), xq) and np.array_equal(s.cpu().numpy(), xs)
        # the experts of every token
        logits, r = take("int8_linear"), take("expert_route")
        ref = product(xq, xs, b.router)
        close(logits, ref, tolerance(ref, F32))
        ids, w, perm, offsets, place = E.route(back(logits), top)
        for got, want in ((r.ids, ids), (r.perm, perm), (r.offsets, offsets), (r.place, place)):
            assert np.array_equal(got.cpu().numpy(), want)
        close(r.weights, w, np.abs(w) * 2.0 ** -18)
        # the shared half
        half, shared = take("int8_gated"), take("int8_linear")
        (gq, gs), (uq, us) = weights(b.gated)
        gv, u = E.product(xq, xs, gq[0], gs[0])[0], E.product(xq, xs, uq[0], us[0])[0]
        ref = E.gate(gv, u, "silu")
        close(half, ref, tolerance(ref, BF, gv, u, "silu"))
        ref = product(*E.quantize(back(half)), b.down)
        close(shared, ref, tolerance(ref, BF))
        # the experts' halves, grouped, and back to the tokens
        half, rows = take("expert_gated"), take("expert_linear")
        ref, gv, u = reference(xq, xs, weights(b.expert_gated), offsets, perm, "silu")
        close(half, ref, tolerance(ref, BF, gv, u, "silu"))
        ref, _, _ = reference(*E.quantize(back(half)), weights(b.expert_down), offsets, np.arange(t * top), None)
        close(rows, ref, tolerance(ref, BF))
        out = take("expert_combine")
        ref, mags = E.combine(back(rows), back(r.weights), place, back(shared))
        close(out, ref, mags * (top + 1) * 2.0 ** -24 + np.abs(ref) * 2.0 ** -8 + 1e-30)
    _, h = take("block_norm")
    check_norm(h, residual + back(out), final)
    logits, said = take("int8_linear"), take("token_logprobs")
    ref = product(*E.quantize(back(h)), head)
    close(logits, ref, tolerance(ref, BF))
    logprob, _, rank, ids, _ = D.token_logprobs(back(logits), tokens.cpu().numpy(), 5, 1.0)
    close(said.logprob, logprob, 2.0 ** -16 + 2.0 ** -21 * np.abs(logprob))
    assert np.array_equal(said.rank.cpu().numpy(), rank) and np.array_equal(said.top_ids.cpu().numpy(), ids)
    assert result is said and not any(made.values())
