"""Scoring tokens through feed-forward blocks that mix the two kinds of weights: the gated half and the output head at a
fixed 8 bits, the down projection in routed bit slices.  The score (log probability of the next tokens) says what a slice
budget costs, which is what a mixed-precision choice is made on.

    python examples/score_block.py [--tokens 256] [--hidden 1024] [--ffn 2816] [--vocab 8000] [--blocks 2]

Random weights stand in for a model; one pass per budget:
  y, q, s = block_norm(block output, residual, ..., quantized=True)   the norm after a block and before the next
  u = fp8_gated(gate and up weights, q, s)                           silu(g) * u in one kernel
  d = linear(down weight in slices, u, routed)                       or fp8_linear for the 8-bit reference
  logits = fp8_linear(head, h);  token_logprobs(logits, next tokens, top=5)
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


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 256), ("hidden", 1024), ("ffn", 2816), ("vocab", 8000), ("blocks", 2)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    blocks, head, final, table = build(a.hidden, a.ffn, a.vocab, a.blocks)
    g = torch.Generator(device=DEV).manual_seed(1)
    tokens = torch.randint(0, a.vocab, (a.tokens + 1,), generator=g, device=DEV)
    x = table[tokens[:-1]]
    # what the 8-bit stack itself would say next: the text that the slice budgets are scored on
    said = score(blocks, head, final, x, tokens[1:], 0).top_ids[:, 0].to(torch.int64)
    for budget in (0, 3, 2, 1):
        r = score(blocks, head, final, x, said, budget)
        name = f"{2 * budget} bits" if budget else "8-bit floats"
        print(f"down projection in {name}: perplexity {math.exp(-float(r.logprob.mean())):.4f}, "
              f"entropy {float(r.entropy.mean()):.4f}, rank 1 for {float((r.rank == 1).float().mean()):.1%}")


if __name__ == "__main__":
    main()
