"""Workloads of the 8-bit integer linear and of the expert operators beside the routed bit-sliced linear.

Four operators, each in two forms that take the same prepared inputs: the plain form (elementary torch operations) and, with
`own` set, the call a user makes of token_adaptive_bit_amd.api.

- linear:  y = sx[t] sw[i] sum_k xq[t][k] wq[i][k], W in 8-bit integers with one float32 scale per output, x quantized within
           the call to 8-bit integers with one scale per token; or the gated half silu(x . Wg^T) * (x . Wu^T) of two.
- route:   each token's top experts from its logits with their weights, and the token copies grouped by expert (stable):
           ids, weights, perm (token of a grouped row), offsets (first row of each expert), place (row of a token's copy).
- experts: the product (or the gated half) of ragged groups of rows, each with its expert's 8-bit integer weight; rows are
           tokens taken through perm (what an expert block reads first), or grouped rows as they lie (what it reads last).
- combine: y[t] = residual[t] + sum_j weights[t][j] rows[place[t][j]].

listed() are the workloads that stand for the range, draw() samples it; work() is the traffic and arithmetic that one pass
cannot do without; exact() is the definition in float64.
"""
import math

import torch

own = False

DEV = "cuda:0"
CODE_MAX = 127.0
AMAX_FLOOR = 2.0 ** -96  # smallest row maximum a scale is made from (a row of zeros stays finite)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token through a square projection: a few microseconds of weight traffic, latency counts
        {"name": "linear t1 5120x5120", "op": "linear", "t": 1, "n": 5120, "k": 5120, "gated": False, "dtype": "bf16"},
        # a ragged chunk of a prompt through a gated half whose sizes are no multiple of any tile, in float32
        {"name": "linear t333 gated 4100x1000", "op": "linear", "t": 333, "n": 4100, "k": 1000, "gated": True, "dtype": "f32"},
        # a long prompt through the down projection: matrix instruction bound
        {"name": "linear t4096 3584x18944", "op": "linear", "t": 4096, "n": 3584, "k": 18944, "gated": False, "dtype": "bf16"},
        # one token choosing its experts: latency
        {"name": "route t1 e64 top6", "op": "route", "t": 1, "e": 64, "top": 6, "score": "softmax", "normalize": True,
         "masked": False, "dtype": "f32"},
        # a prompt choosing its experts, some ruled out, some tokens padding
        {"name": "route t4096 e128 top8", "op": "route", "t": 4096, "e": 128, "top": 8, "score": "softmax", "normalize": True,
         "masked": True, "dtype": "f32"},
        # one token through the gated halves of its experts: their weights' bytes
        {"name": "experts t1 gated e64 top6 1408x2048", "op": "experts", "t": 1, "e": 64, "top": 6, "n": 1408, "k": 2048,
         "gated": True, "gather": True, "dtype": "bf16"},
        # a decode batch through the down projections: nearly every expert is read for a row or two
        {"name": "experts t32 e128 top8 2048x768", "op": "experts", "t": 32, "e": 128, "top": 8, "n": 2048, "k": 768,
         "gated": False, "gather": False, "dtype": "bf16"},
        # a ragged chunk, odd sizes, float32
        {"name": "experts t200 e40 top3 1000x1100", "op": "experts", "t": 200, "e": 40, "top": 3, "n": 1000, "k": 1100,
         "gated": False, "gather": True, "dtype": "f32"},
        # a prompt through the gated halves of many small experts
        {"name": "experts t4096 gated e128 top8 1536x4096", "op": "experts", "t": 4096, "e": 128, "top": 8, "n": 1536, "k": 4096,
         "gated": True, "gather": True, "dtype": "bf16"},
        # a long prompt through the down projections of few large experts
        {"name": "experts t8192 e8 top2 4096x14336", "op": "experts", "t": 8192, "e": 8, "top": 2, "n": 4096, "k": 14336,
         "gated": False, "gather": False, "dtype": "bf16"},
        # a decode batch's expert outputs back into the residual stream: latency
        {"name": "combine t7 n2050 top6", "op": "combine", "t": 7, "n": 2050, "top": 6, "dtype": "bf16"},
        # a prompt's: memory
        {"name": "combine t8192 n4096 top8", "op": "combine", "t": 8192, "n": 4096, "top": 8, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, v, step):
    """Mostly a multiple of step, as model widths are; one in three left as drawn."""
    return v if rng.random() < 1 / 3 else max(step, v // step * step)


def draw(rng):
    op = rng.choice(["linear", "linear", "route", "experts", "experts", "experts", "combine"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "linear":
        gated = rng.random() < 0.35
        n, k = _odd(rng, _log_int(rng, 256, 19000), 64), _odd(rng, _log_int(rng, 256, 19000), 128)
        t = min(_log_int(rng, 1, 4096), max(1, int(2.7e11 / (n * k * (1 + gated)))))
        return {"op": op, "t": t, "n": n, "k": k, "gated": gated, "dtype": dtype}
    if op == "route":
        e = _odd(rng, _log_int(rng, 4, 512), 4)
        return {"op": op, "t": _log_int(rng, 1, 4096), "e": e, "top": rng.randint(1, min(8, e)),
                "score": rng.choice(["softmax", "softmax", "sigmoid"]), "normalize": rng.random() < 0.7,
                "masked": rng.random() < 0.5, "dtype": dtype}
    if op == "experts":
        e, gated = _log_int(rng, 4, 256), rng.random() < 0.5
        n, k = _odd(rng, _log_int(rng, 256, 14400), 64), _odd(rng, _log_int(rng, 256, 14400), 128)
        e = max(4, min(e, int(1.2e9 / (n * k * (1 + gated)))))
        top = rng.randint(1, min(8, e))
        t = min(_log_int(rng, 1, 8192), max(1, int(9.0e11 / (n * k * (1 + gated) * top))), max(1, (1 << 26) // (max(n, k) * top)))
        return {"op": op, "t": t, "e": e, "top": top, "n": n, "k": k, "gated": gated, "gather": gated or rng.random() < 0.4,
                "dtype": dtype}
    n, top = _odd(rng, _log_int(rng, 128, 16384), 64), rng.randint(1, 8)
    t = min(_log_int(rng, 1, 8192), max(1, (1 << 28) // (n * top * (2 if dtype == "f32" else 1))))
    return {"op": op, "t": t, "n": n, "top": top, "dtype": dtype}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFF)


def _activations(t, k, dtype, g):
    """Normal values with a few channels 20 times as large, as hidden states have them."""
    x = torch.randn(t, k, generator=g, device=DEV)
    x[:, torch.randint(0, k, (max(1, k // 512),), generator=g, device=DEV)] *= 20.0
    return x.to(TYPES[dtype])


def _integer_weight(shape, g):
    """A checkpoint's 8-bit integer weight [..., n, k] and the float32 scale of every output [..., n]: rows of normal values,
    the largest of a row at 127."""
    codes = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16).mul_(CODE_MAX / 3.6).round_().clamp_(-CODE_MAX, CODE_MAX)
    scale = torch.rand(shape[:-1], generator=g, device=DEV).add_(0.5).mul_(0.7 * 3.6 / (CODE_MAX * math.sqrt(shape[-1])))
    return codes.to(torch.int8), scale


def _logits(t, e, g):
    """Router logits: some experts more popular than others."""
    return torch.randn(t, e, generator=g, device=DEV).mul_(1.5) + 0.7 * torch.randn(e, generator=g, device=DEV)


def _inputs(case, seed):
    g, op, t = _gen(seed), case["op"], case["t"]
    if op == "linear":
        s = {"x": _activations(t, case["k"], case["dtype"], g), "w": _integer_weight((case["n"], case["k"]), g)}
        if case["gated"]:
            s["w2"] = _integer_weight((case["n"], case["k"]), g)
        return s
    if op == "route":
        z, e = _logits(t, case["e"], g), case["e"]
        if case["masked"]:                                         # a tenth of the experts is away, some tokens are padding
            z[:, torch.rand(e, generator=g, device=DEV) < 0.1] = float("-inf")
            z[torch.rand(t, generator=g, device=DEV) < 0.05] = float("-inf")
        return {"logits": z.to(TYPES[case["dtype"]])}
    if op == "experts":
        e, n, k, top = case["e"], case["n"], case["k"], case["top"]
        chosen = _logits(t, e, g).topk(top, dim=1).indices.flatten()
        order = torch.argsort(chosen, stable=True)
        counts = torch.bincount(chosen, minlength=e)
        s = {"perm": (order // top).to(torch.int32), "counts": counts.tolist(),
             "offsets": torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32),
             "x": _activations(t if case["gather"] else t * top, k, case["dtype"], g), "w": _integer_weight((e, n, k), g)}
        if case["gated"]:
            s["w2"] = _integer_weight((e, n, k), g)
        return s
    n, top = case["n"], case["top"]
    rows = torch.randn(t * top, n, generator=g, device=DEV).to(TYPES[case["dtype"]])
    place = torch.randperm(t * top, generator=g, device=DEV).view(t, top).to(torch.int32)
    place[torch.rand(t, generator=g, device=DEV) < 0.05] = -1      # padding: tokens without experts
    weights = torch.rand(t, top, generator=g, device=DEV)
    weights = torch.where(place >= 0, weights / weights.sum(1, keepdim=True), 0.0)
    return {"rows": rows, "place": place, "weights": weights, "residual": _activations(t, n, case["dtype"], g)}


def prepare(case, seed):
    state = dict(_inputs(case, seed), case=dict(case))
    if own and case["op"] in ("linear", "experts"):
        from token_adaptive_bit_amd import api
        w, s = state.pop("w")
        one, two = (api.int8_pack, api.int8_pack_gated) if case["op"] == "linear" else (api.expert_pack, api.expert_pack_gated)
        if case["gated"]:
            w2, s2 = state.pop("w2")
            state["packed"] = two(w, w2, s, s2)
        else:
            state["packed"] = one(w, s)
    return state


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    from token_adaptive_bit_amd import api
    case = state["case"]
    if case["op"] == "linear":
        return (api.int8_gated if case["gated"] else api.int8_linear)(state["packed"], state["x"])
    if case["op"] == "route":
        return tuple(api.expert_route(state["logits"], case["top"], score=case["score"], normalize=case["normalize"]))
    if case["op"] == "experts":
        rows = state["perm"] if case["gather"] else None
        return (api.expert_gated if case["gated"] else api.expert_linear)(state["packed"], state["x"], state["offsets"], rows)
    return api.expert_combine(state["rows"], state["weights"], state["place"], state["residual"])


def _quantize_plain(x):
    """x [t, k]: integer values [t, k] float32 and the scale of every token [t, 1]; the factor 127 / max in 64 bits, rounded
    once, so that values next to a border fall on the side that the definition gives them."""
    x = x.float()
    amax = x.abs().amax(dim=1, keepdim=True).clamp_min(AMAX_FLOOR).double()
    return torch.round(x * (CODE_MAX / amax).float()), (amax / CODE_MAX).float()


def _product_plain(q, scale, w, ws):
    return (q @ w.float().t()) * scale * ws


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "linear":
        q, scale = _quantize_plain(state["x"])
        y = _product_plain(q, scale, *state["w"])
        if case["gated"]:
            y = y / (1.0 + torch.exp(-y)) * _product_plain(q, scale, *state["w2"])
        return y.to(state["x"].dtype)
    if op == "route":
        return _route_plain(state["logits"].float(), case)
    if op == "experts":
        q, scale = _quantize_plain(state["x"])
        if case["gather"]:
            at = state["perm"].long()
            q, scale = q[at], scale[at]
        (w, ws), out, first = state["w"], [], 0
        for e, count in enumerate(state["counts"]):
            if count == 0:
                continue
            rows = slice(first, first + count)
            first += count
            y = _product_plain(q[rows], scale[rows], w[e], ws[e])
            if case["gated"]:
                w2, s2 = state["w2"]
                y = y / (1.0 + torch.exp(-y)) * _product_plain(q[rows], scale[rows], w2[e], s2[e])
            out.append(y)
        return torch.cat(out).to(state["x"].dtype)
    rows, place, weights = state["rows"], state["place"].long(), state["weights"]
    y = state["residual"].float()
    for j in range(case["top"]):
        part = rows[place[:, j].clamp_min(0)].float() * weights[:, j, None]
        y = y + torch.where(place[:, j, None] >= 0, part, 0.0)
    return y.to(rows.dtype)


def _route_plain(z, case):
    (t, e), top = z.shape, case["top"]
    bits = (z + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)       # orders as the values do
    index = torch.arange(e, device=z.device)
    chosen = ((key << 32) + (e - 1 - index)).topk(top, dim=1).indices          # equal values: the lowest index first
    best = z.gather(1, chosen)
    there = best > float("-inf")
    if case["score"] == "softmax":
        m = best[:, :1]
        scores = torch.where(there, torch.exp(best - m), 0.0)
        total = scores if case["normalize"] else torch.where(z > float("-inf"), torch.exp(z - m), 0.0)
        weights = torch.where(there, scores / total.sum(1, keepdim=True), 0.0)
    else:
        weights = torch.where(there, 1.0 / (1.0 + torch.exp(-best)), 0.0)
        if case["normalize"]:
            weights = torch.where(there, weights / weights.sum(1, keepdim=True), 0.0)
    ids = torch.where(there, chosen, -1)
    flat = torch.where(there, chosen, e).flatten()                             # places without an expert go last
    order = torch.argsort(flat, stable=True)
    counts = (flat[:, None] == index).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    position = torch.arange(t * top, device=z.device)
    perm = torch.where(position < offsets[e], order // top, -1)
    place = torch.where(flat < e, torch.empty_like(order).scatter_(0, order, position), -1)
    i32 = torch.int32
    return ids.to(i32), weights, perm.to(i32), offsets.to(i32), place.view(t, top).to(i32)


def work(case):
    op, t, size = case["op"], case["t"], 2 if case["dtype"] == "bf16" else 4
    if op == "linear":
        n, k, two = case["n"], case["k"], 1 + case["gated"]
        return {"bytes": t * k * size + two * n * (k + 4) + t * n * size, "flops": 2 * two * t * n * k}
    if op == "route":
        e, top = case["e"], case["top"]
        return {"bytes": t * e * size + 16 * t * top + 4 * (e + 1), "flops": 4 * t * e}
    if op == "experts":
        e, n, k, top, two = case["e"], case["n"], case["k"], case["top"], 1 + case["gated"]
        read = e * (1.0 - (1.0 - top / e) ** t)          # experts that have a row, were they equally popular
        rows = t if case["gather"] else t * top
        return {"bytes": int(rows * k * size + read * two * n * (k + 4) + t * top * n * size) + 4 * (t * top + e + 1),
                "flops": 2 * two * t * top * n * k}
    n, top = case["n"], case["top"]
    return {"bytes": (top + 2) * t * n * size + 8 * t * top, "flops": 2 * t * top * n}


def _integers64(x):
    """Integer values and scales of x [t, k] by the definition: factor, scale and product rounded to float32 once each."""
    x = x.to(torch.float64)
    top = x.abs().max(dim=1, keepdim=True).values.clamp_min(AMAX_FLOOR)
    return (x * (CODE_MAX / top).float().to(x.dtype)).float().to(x.dtype).round(), (top / CODE_MAX).float().to(x.dtype)


def exact(case, seed):
    s, f64, op = _inputs(case, seed), torch.float64, case["op"]
    if op == "linear":
        q, scale = _integers64(s["x"])
        outs = [torch.mm(q, w.to(f64).t().contiguous()) * (scale * ws.to(f64)) for w, ws in [s[name] for name in ("w", "w2") if name in s]]
        return outs[0] if len(outs) == 1 else outs[0] * torch.sigmoid(outs[0]) * outs[1]
    if op == "route":
        z = s["logits"].to(f64)
        t, e, top = case["t"], case["e"], case["top"]
        values, ids = (part[:, :top] for part in z.sort(dim=1, descending=True, stable=True))
        away = torch.isneginf(values)
        score = torch.sigmoid(values) if case["score"] == "sigmoid" else torch.softmax(z, 1).gather(1, ids)
        score = score.masked_fill(away, 0.0)
        if case["normalize"]:
            score = (score / score.sum(1, keepdim=True)).masked_fill(away, 0.0)
        return None, score, None, None, None
    if op == "experts":
        q, scale = _integers64(s["x"])
        parts, first, perm = [], 0, s["perm"].long()
        for e, count in enumerate(s["counts"]):
            at = perm[first : first + count] if case["gather"] else torch.arange(first, first + count, device=DEV)
            first += count
            outs = [torch.mm(q[at], w[e].to(f64).t().contiguous()) * (scale[at] * ws[e].to(f64))
                    for w, ws in [s[name] for name in ("w", "w2") if name in s]]
            parts.append(outs[0] if len(outs) == 1 else outs[0] * torch.sigmoid(outs[0]) * outs[1])
        return torch.cat(parts)
    y, place = s["residual"].to(f64), s["place"].long()
    padded = torch.cat([s["rows"], s["rows"].new_zeros(1, case["n"])])          # row -1: zeros
    for lo in range(0, case["t"], 1024):
        band = slice(lo, lo + 1024)
        taken = padded[place[band]].to(f64)
        y[band] += (taken * s["weights"][band].to(f64).unsqueeze(2)).sum(1)
    return y
