"""Scoring tokens through feed-forward blocks that mix the two kinds of weights: the gated half and the output head at a
fixed 8 bits, the down projection in routed bit slices.  The score (log probability of the next tokens) says what a slice
budget costs, which is what a mixed-precision choice is made on.

    python examples/score_block.py [--tokens 256] [--hidden 1024] [--ffn 2816] [--vocab 8000] [--blocks 2] [--experts 0]

Random weights stand in for a model; one pass per budget:
  y, q, s = block_norm(block output, residual, ..., quantized=True)   the norm after a block and before the next
  u = fp8_gated(gate and up weights, q, s)                           silu(g) * u in one kernel
  d = linear(down weight in slices, u, routed)                       or fp8_linear for the 8-bit reference
  logits = fp8_linear(head, h);  token_logprobs(logits, next tokens, top=5)

With --experts the blocks are of experts in 8-bit integers beside a shared half, and the score says what fewer experts a
token cost:
  q, s = int8_quantize(h)                                            once for all that read the block's input
  r = expert_route(int8_linear(router, q, s), top)                   experts, weights, and the copies grouped by expert
  shared = int8_linear(down, int8_gated(gate and up weights, q, s))
  u = expert_gated(experts' gate and up weights, q, r.offsets, r.perm, s)
  out = expert_combine(expert_linear(experts' down, u, r.offsets), r.weights, r.place, shared)
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from token_adaptive_bit_amd import api  # noqa: E402

DEV = "cuda:0"


class Block:
    def __init__(self, hidden: int, ffn: int, g: torch.Generator):
        def w(n, k):
            return (torch.randn(n, k, generator=g, device=DEV) / math.sqrt(k)).bfloat16()

        self.pre = 1 + 0.1 * torch.randn(hidden, generator=g, device=DEV)
        self.post = 1 + 0.1 * torch.randn(hidden, generator=g, device=DEV)
        self.gate = torch.full((hidden,), 0.5, device=DEV)       # layer scale of the block into the residual stream
        self.gated = api.fp8_pack_gated(w(ffn, hidden), w(ffn, hidden))
        down = w(hidden, ffn)
        self.down8 = api.fp8_pack(down)
        self.down = api.pack(down, group=128, slices=3)


def score(blocks, head, final, embedded, targets, budget: int, top: int = 5) -> api.TokenLogprobs:
    """Log probabilities of `targets` after the embedded tokens, with the down projections at `budget` slices (0: 8 bits)."""
    t = embedded.shape[0]
    if budget:
        perm, offsets = api.regroup(torch.full((t,), budget, dtype=torch.int32, device=DEV), 3)
    residual, out, last = embedded, None, None
    for b in blocks:
        if out is None:      # before the first block: a norm only
            residual, q, s = api.block_norm(residual, None, pre=b.pre, quantized=True)
        else:                # after the last block and before this one
            residual, q, s = api.block_norm(out, residual, pre=b.pre, post=last.post, gate=last.gate, quantized=True)
        u = api.fp8_gated(b.gated, q, s)
        out = api.linear(b.down, u, perm, offsets) if budget else api.fp8_linear(b.down8, u)
        last = b
    _, q, s = api.block_norm(out, residual, pre=final, post=last.post, gate=last.gate, quantized=True)
    return api.token_logprobs(api.fp8_linear(head, q, s), targets, top=top)


def build(hidden: int, ffn: int, vocab: int, blocks: int, seed: int = 0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    stack = [Block(hidden, ffn, g) for _ in range(blocks)]
    table = torch.randn(vocab, hidden, generator=g, device=DEV).bfloat16()
    head = torch.randn(vocab, hidden, generator=g, device=DEV) * (3 / math.sqrt(hidden))
    return stack, api.fp8_pack(head.bfloat16()), torch.ones(hidden, device=DEV), table


class ExpertBlock:
    def __init__(self, hidden: int, ffn: int, experts: int, g: torch.Generator):
        def w(*shape):
            return (torch.randn(*shape, generator=g, device=DEV) / math.sqrt(shape[-1])).bfloat16()

        self.pre = 1 + 0.1 * torch.randn(hidden, generator=g, device=DEV)
        self.router = api.int8_pack(w(experts, hidden))
        self.gated = api.int8_pack_gated(w(ffn, hidden), w(ffn, hidden))
        self.down = api.int8_pack(w(hidden, ffn))
        self.expert_gated = api.expert_pack_gated(w(experts, ffn, hidden), w(experts, ffn, hidden))
        self.expert_down = api.expert_pack(w(experts, hidden, ffn))


def score_experts(blocks, head, final, embedded, targets, experts: int, top: int = 5) -> api.TokenLogprobs:
    """Log probabilities of `targets` after the embedded tokens, with `experts` experts a token."""
    residual, out = embedded, None
    for b in blocks:
        if out is None:
            residual, h = api.block_norm(residual, None, pre=b.pre)
        else:
            residual, h = api.block_norm(out, residual, pre=b.pre)
        q, s = api.int8_quantize(h)
        r = api.expert_route(api.int8_linear(b.router, q, s, out_dtype=torch.float32), experts)
        shared = api.int8_linear(b.down, api.int8_gated(b.gated, q, s))
        u = api.expert_gated(b.expert_gated, q, r.offsets, r.perm, s)
        out = api.expert_combine(api.expert_linear(b.expert_down, u, r.offsets), r.weights, r.place, shared)
    _, h = api.block_norm(out, residual, pre=final)
    return api.token_logprobs(api.int8_linear(head, h), targets, top=top)


def build_experts(hidden: int, ffn: int, vocab: int, blocks: int, experts: int, seed: int = 0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    stack = [ExpertBlock(hidden, ffn, experts, g) for _ in range(blocks)]
    table = torch.randn(vocab, hidden, generator=g, device=DEV).bfloat16()
    head = torch.randn(vocab, hidden, generator=g, device=DEV) * (3 / math.sqrt(hidden))
    return stack, api.int8_pack(head.bfloat16()), torch.ones(hidden, device=DEV), table


def report(name: str, r: api.TokenLogprobs) -> None:
    print(f"{name}: perplexity {math.exp(-float(r.logprob.mean())):.4f}, "
          f"entropy {float(r.entropy.mean()):.4f}, rank 1 for {float((r.rank == 1).float().mean()):.1%}")


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 256), ("hidden", 1024), ("ffn", 2816), ("vocab", 8000), ("blocks", 2), ("experts", 0)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    if a.experts:
        blocks, head, final, table = build_experts(a.hidden, a.ffn, a.vocab, a.blocks, a.experts)
    else:
        blocks, head, final, table = build(a.hidden, a.ffn, a.vocab, a.blocks)
    g = torch.Generator(device=DEV).manual_seed(1)
    tokens = torch.randint(0, a.vocab, (a.tokens + 1,), generator=g, device=DEV)
    x = table[tokens[:-1]]
    if a.experts:
        # the text is what the stack says with all the experts that are tried
        tops = [n for n in (8, 4, 2, 1) if n <= a.experts]
        said = score_experts(blocks, head, final, x, tokens[1:], tops[0]).top_ids[:, 0].to(torch.int64)
        for n in tops:
            report(f"{n} of {a.experts} experts a token", score_experts(blocks, head, final, x, said, n))
        return
    # what the 8-bit stack itself would say next: the text that the slice budgets are scored on
    said = score(blocks, head, final, x, tokens[1:], 0).top_ids[:, 0].to(torch.int64)
    for budget in (0, 3, 2, 1):
        name = f"{2 * budget} bits" if budget else "8-bit floats"
        report(f"down projection in {name}", score(blocks, head, final, x, said, budget))


if __name__ == "__main__":
    main()
