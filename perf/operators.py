"""Workloads of the dense operators that stand beside the routed bit-sliced linear.

Four operators, each in two forms that take the same prepared inputs: the plain form (elementary torch operations in
float32) and, with `own` set, the call a user makes of token_adaptive_bit_amd.api.

- linear:   y = x . W^T, W in e4m3 codes with one float32 scale per 128 x 128 block, x quantized within the call to e4m3
            with one scale per token and 128 inputs.
- gated:    y = silu(x . Wg^T) * (x . Wu^T) on two such weights (the first half of a gated feed-forward block).
- norm:     y = a * residual + b * gate * post(x), h = pre(y): the norm after a block, its gate and scale into the
            residual stream, and the norm before the next block, optionally with h as e4m3 codes and scales.
- logprobs: log probability, entropy and rank of given tokens from logits, with the top alternatives.

listed() are the workloads that stand for the range, draw() samples it; work() is the traffic and arithmetic that one pass
cannot do without; exact() is the definition in float64.
"""
import math

import torch

own = False

DEV = "cuda:0"
BLOCK = 128              # inputs per activation scale, and both sides of a weight's scale block
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -96  # smallest block maximum a scale is made from (an all-zero block stays finite)
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token through a square projection: the call is a few microseconds of weight traffic, latency counts
        {"name": "linear t1 5120x5120", "op": "linear", "t": 1, "n": 5120, "k": 5120, "dtype": "bf16"},
        # a decode batch through the widest weight of the benchmark: weight traffic bound
        {"name": "linear t16 18944x3584", "op": "linear", "t": 16, "n": 18944, "k": 3584, "dtype": "bf16"},
        # a ragged chunk of a prompt on sizes that are no multiple of any tile, float32 activations
        {"name": "linear t333 4100x1000", "op": "linear", "t": 333, "n": 4100, "k": 1000, "dtype": "f32"},
        # a long prompt through the down projection: matrix instruction bound
        {"name": "linear t4096 3584x18944", "op": "linear", "t": 4096, "n": 3584, "k": 18944, "dtype": "bf16"},
        # one token through the gated half of a feed-forward block
        {"name": "gated t1 13824x5120", "op": "gated", "t": 1, "n": 13824, "k": 5120, "dtype": "bf16"},
        # a prompt through the gated half
        {"name": "gated t2048 11008x4096", "op": "gated", "t": 2048, "n": 11008, "k": 4096, "dtype": "bf16"},
        # decode: one token between two blocks, handed on as 8-bit codes
        {"name": "norm t1 k5120 q", "op": "norm", "t": 1, "k": 5120, "dtype": "bf16", "kind": "rms", "post": True,
         "gate": "none", "quantized": True},
        # a small batch at an odd width, layer norm, a gate per token and channel, float32
        {"name": "norm t77 k1531 layer", "op": "norm", "t": 77, "k": 1531, "dtype": "f32", "kind": "layer",
         "post": False, "gate": "full", "quantized": False},
        # a long prompt between two blocks, both norms and a gate per channel
        {"name": "norm t16384 k4096", "op": "norm", "t": 16384, "k": 4096, "dtype": "bf16", "kind": "rms", "post": True,
         "gate": "channel", "quantized": False},
        # one sampled token reported with its alternatives
        {"name": "logprobs t1 v131072", "op": "logprobs", "t": 1, "v": 131072, "dtype": "f32", "top": 20},
        # a decode batch over an odd vocabulary
        {"name": "logprobs t64 v50021", "op": "logprobs", "t": 64, "v": 50021, "dtype": "bf16", "top": 5},
        # scoring a prompt (perplexity) with a few alternatives per position
        {"name": "logprobs t2048 v128000", "op": "logprobs", "t": 2048, "v": 128000, "dtype": "bf16", "top": 8},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, v, step):
    """Mostly a multiple of step, as model widths are; one in three left as drawn."""
    return v if rng.random() < 1 / 3 else max(step, v // step * step)


def draw(rng):
    op = rng.choice(["linear", "gated", "norm", "logprobs"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("linear", "gated"):
        most = 19000 if op == "linear" else 14000
        n, k = _odd(rng, _log_int(rng, 256, most), 64), _odd(rng, _log_int(rng, 256, most), 128)
        t = min(_log_int(rng, 1, 4096), max(1, int(2.0e11 / (n * k * (2 if op == "gated" else 1)))))
        return {"op": op, "t": t, "n": n, "k": k, "dtype": dtype}
    if op == "norm":
        k = _odd(rng, _log_int(rng, 64, 20000), 128)
        t = min(_log_int(rng, 1, 16384), max(1, (64 << 20) // k))
        return {"op": op, "t": t, "k": k, "dtype": dtype, "kind": rng.choice(["rms", "rms", "layer"]),
                "post": rng.random() < 0.6, "gate": rng.choice(["none", "channel", "token", "full"]),
                "quantized": rng.random() < 0.4}
    v = _odd(rng, _log_int(rng, 1000, 262144), 128)
    t = min(_log_int(rng, 1, 4096), max(1, (128 << 20) // v))
    return {"op": op, "t": t, "v": v, "dtype": dtype, "top": rng.choice([0, 1, 5, 8, 20])}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFF)


def _activations(t, k, dtype, g):
    """Normal values with a few channels 20 times as large, as hidden states have them."""
    x = torch.randn(t, k, generator=g, device=DEV)
    x[:, torch.randint(0, k, (max(1, k // 512),), generator=g, device=DEV)] *= 20.0
    return x.to(TYPES[dtype])


def _quantized_weight(n, k, g):
    """A checkpoint's 8-bit weight: e4m3 codes [n, k] and the float32 scale of every 128 x 128 block."""
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    w = torch.zeros(nb * BLOCK, kb * BLOCK, device=DEV)
    w[:n, :k] = torch.randn(n, k, generator=g, device=DEV).mul_(0.7 / math.sqrt(k))
    w = w.view(nb, BLOCK, kb, BLOCK)
    amax = w.abs().amax(dim=(1, 3)).clamp_min_(AMAX_FLOOR)
    codes = (w * (E4M3_MAX / amax)[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:n, :k].to(F8).contiguous()
    return codes, amax / E4M3_MAX


def _inputs(case, seed):
    g, op = _gen(seed), case["op"]
    if op in ("linear", "gated"):
        s = {"x": _activations(case["t"], case["k"], case["dtype"], g), "w": _quantized_weight(case["n"], case["k"], g)}
        if op == "gated":
            s["w2"] = _quantized_weight(case["n"], case["k"], g)
        return s
    t, dt = case["t"], TYPES[case["dtype"]]
    if op == "norm":
        k = case["k"]
        s = {"x": _activations(t, k, case["dtype"], g), "residual": _activations(t, k, case["dtype"], g)}
        s["pre"] = 1.0 + 0.1 * torch.randn(k, generator=g, device=DEV)
        s["post"] = 1.0 + 0.1 * torch.randn(k, generator=g, device=DEV) if case["post"] else None
        shape = {"none": None, "channel": (k,), "token": (t,), "full": (t, k)}[case["gate"]]
        s["gate"] = None
        if shape:
            s["gate"] = torch.sigmoid(torch.randn(shape, generator=g, device=DEV))
            if case["gate"] == "full":
                s["gate"] = s["gate"].to(dt)
        return s
    v = case["v"]
    z = torch.randn(t, v, generator=g, device=DEV).mul_(2.5)
    rows = torch.arange(t, device=DEV)
    z[rows, torch.randint(0, v, (t,), generator=g, device=DEV)] += 12.0 * torch.rand(t, generator=g, device=DEV)
    masked = torch.rand(t, generator=g, device=DEV) < 0.3        # rows under a grammar: half their tokens ruled out
    z[:, : v // 2].masked_fill_(masked[:, None], float("-inf"))
    targets = torch.randint(v // 2, v, (t,), generator=g, device=DEV)
    targets[torch.rand(t, generator=g, device=DEV) < 0.05] = -1   # padding
    return {"logits": z.to(dt), "targets": targets}


def prepare(case, seed):
    state = dict(_inputs(case, seed), case=dict(case))
    if own and case["op"] in ("linear", "gated"):
        from token_adaptive_bit_amd import api
        w, s = state["w"]
        state["packed"] = api.fp8_pack_gated(w, state["w2"][0], s, state["w2"][1]) if "w2" in state else api.fp8_pack(w, s)
    return state


RESIDUAL_SCALE, GATE_SCALE, EPS, INV_TEMPERATURE = 0.9, 1.1, 1e-6, 1.0 / 0.8


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    from token_adaptive_bit_amd import api
    case = state["case"]
    if case["op"] == "linear":
        return api.fp8_linear(state["packed"], state["x"], out_dtype=torch.bfloat16)
    if case["op"] == "gated":
        return api.fp8_gated(state["packed"], state["x"], out_dtype=torch.bfloat16)
    if case["op"] == "norm":
        return api.block_norm(state["x"], state["residual"], pre=state["pre"], post=state["post"], gate=state["gate"],
                              residual_scale=RESIDUAL_SCALE, gate_scale=GATE_SCALE, eps=EPS, kind=case["kind"],
                              quantized=case["quantized"])
    return api.token_logprobs(state["logits"], state["targets"], top=case["top"], inv_temperature=INV_TEMPERATURE)


def _quantize_plain(x):
    """x [t, k] float32: e4m3 codes [t, k], the float32 scales [ceil(k / 128), t] and the values they stand for."""
    t, k = x.shape
    kb = -(-k // BLOCK)
    xb = torch.nn.functional.pad(x, (0, kb * BLOCK - k)).view(t, kb, BLOCK)
    amax = xb.abs().amax(dim=2).clamp_min(AMAX_FLOOR)
    codes = (xb * (E4M3_MAX / amax)[:, :, None]).to(F8)
    scale = amax / E4M3_MAX
    values = (codes.float() * scale[:, :, None]).view(t, kb * BLOCK)[:, :k]
    return codes.view(t, kb * BLOCK)[:, :k].contiguous(), scale.t().contiguous(), values


def _dequantize_plain(w):
    codes, scale = w
    n, k = codes.shape
    return codes.float() * scale.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]


def _norm_plain(x, weight, kind):
    if kind == "layer":
        x = x - x.mean(dim=1, keepdim=True)
    return x / torch.sqrt(x.square().mean(dim=1, keepdim=True) + EPS) * weight


def _run_plain(state):
    case = state["case"]
    if case["op"] in ("linear", "gated"):
        values = _quantize_plain(state["x"].float())[2]
        y = values @ _dequantize_plain(state["w"]).t()
        if case["op"] == "gated":
            y = y / (1.0 + torch.exp(-y)) * (values @ _dequantize_plain(state["w2"]).t())
        return y.to(torch.bfloat16)
    if case["op"] == "norm":
        dt, gate = state["x"].dtype, state["gate"]
        z = state["x"].float()
        if state["post"] is not None:
            z = _norm_plain(z, state["post"], case["kind"])
        if gate is not None:
            z = z * (gate[:, None] if case["gate"] == "token" else gate.float())
        y = RESIDUAL_SCALE * state["residual"].float() + GATE_SCALE * z
        h = _norm_plain(y, state["pre"], case["kind"])
        if case["quantized"]:
            codes, scale, _ = _quantize_plain(h)
            return y.to(dt), codes, scale
        return y.to(dt), h.to(dt)
    z, targets, top = state["logits"].float(), state["targets"], case["top"]
    t, v = z.shape
    m = z.amax(dim=1, keepdim=True)
    d = (z - m) * INV_TEMPERATURE
    e = torch.exp(d)
    s = e.sum(dim=1)
    log_s = torch.log(s)
    entropy = log_s - torch.where(e > 0, e * d, 0.0).sum(dim=1) / s
    valid = (targets >= 0) & (targets < v)
    at = targets.clamp(0, v - 1)[:, None]
    logprob = torch.where(valid, d.gather(1, at)[:, 0] - log_s, 0.0)
    zt = z.gather(1, at)
    ids = torch.arange(v, device=z.device)
    rank = torch.where(valid, 1 + ((z > zt) | ((z == zt) & (ids < at))).sum(dim=1), 0).to(torch.int32)
    if not top:
        return logprob, entropy, rank
    bits = (z + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)       # orders as the values do
    order = ((key << 32) + (v - 1 - ids)).topk(top, dim=1).indices             # equal values: the lowest index first
    return logprob, entropy, rank, order.to(torch.int32), d.gather(1, order) - log_s[:, None]


def work(case):
    t, size = case["t"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("linear", "gated"):
        n, k, two = case["n"], case["k"], 2 if case["op"] == "gated" else 1
        weight = two * (n * k + 4 * -(-n // BLOCK) * -(-k // BLOCK))
        return {"bytes": t * k * size + weight + 2 * t * n, "flops": 2 * two * t * n * k}
    if case["op"] == "norm":
        k = case["k"]
        gate = {"none": 0, "channel": 4 * k, "token": 4 * t, "full": t * k * size}[case["gate"]]
        h = t * k + 4 * t * -(-k // BLOCK) if case["quantized"] else t * k * size
        return {"bytes": 3 * t * k * size + 4 * k * (2 if case["post"] else 1) + gate + h, "flops": 12 * t * k}
    return {"bytes": t * case["v"] * size + t * (8 + 12 + 8 * case["top"]), "flops": 6 * t * case["v"]}


def exact(case, seed):
    s, f64 = _inputs(case, seed), torch.float64
    if case["op"] in ("linear", "gated"):
        x = s["x"].to(f64)
        xq, xs = _codes64(x)
        xv = (xq * xs.repeat_interleave(BLOCK, 1)[:, : x.shape[1]])
        outs = []
        for codes, scale in [s[name] for name in ("w", "w2") if name in s]:
            out = torch.zeros(x.shape[0], codes.shape[0], dtype=f64, device=DEV)
            for j in range(scale.shape[0]):      # one band of 128 outputs at a time
                rows = slice(j * BLOCK, min((j + 1) * BLOCK, codes.shape[0]))
                band = codes[rows].to(f64) * scale[j].to(f64).repeat_interleave(BLOCK)[: codes.shape[1]]
                out[:, rows] = torch.mm(xv, band.t().contiguous())
            outs.append(out)
        return outs[0] if len(outs) == 1 else outs[0] * torch.sigmoid(outs[0]) * outs[1]
    if case["op"] == "norm":
        def norm(a, w):
            mean = a.mean(1, keepdim=True) if case["kind"] == "layer" else 0.0
            var = (a - mean).pow(2).sum(1, keepdim=True) / a.shape[1]
            return (a - mean) * torch.rsqrt(var + EPS) * w.to(f64)

        branch = s["x"].to(f64) if s["post"] is None else norm(s["x"].to(f64), s["post"])
        if case["gate"] == "token":
            branch = branch * s["gate"].to(f64).unsqueeze(1)
        elif case["gate"] != "none":
            branch = branch * s["gate"].to(f64)
        y = s["residual"].to(f64) * RESIDUAL_SCALE + branch * GATE_SCALE
        h = norm(y, s["pre"])
        if not case["quantized"]:
            return y, h
        q, scale = _codes64(h)
        return y, q, scale.t().contiguous()
    outs = []
    for lo in range(0, case["t"], 256):          # bands of rows: float64 copies of the logits stay small
        z = s["logits"][lo : lo + 256].to(f64) * INV_TEMPERATURE
        logp = torch.log_softmax(z, 1)
        p = logp.exp()
        entropy = -(p * logp.masked_fill(p == 0, 0.0)).sum(1)
        target = s["targets"][lo : lo + 256]
        valid = target >= 0
        logprob = logp.gather(1, target.clamp_min(0).unsqueeze(1)).squeeze(1).masked_fill(~valid, 0.0)
        outs.append((logprob, entropy, logp.sort(dim=1, descending=True, stable=True).values[:, : case["top"]]))
    logprob, entropy, best = (torch.cat(parts) for parts in zip(*outs))
    return (logprob, entropy, None, None, best) if case["top"] else (logprob, entropy, None)


def _codes64(x):
    """Codes and scales of x [t, k] float64 per token and 128 inputs, by the definition (scales rounded to float32)."""
    t, k = x.shape
    codes, scales = torch.empty_like(x), []
    for j in range(0, k, BLOCK):
        part = x[:, j : j + BLOCK]
        top = part.abs().max(dim=1).values.clamp_min(AMAX_FLOOR)
        codes[:, j : j + BLOCK] = (part * (E4M3_MAX / top).float().to(x.dtype).unsqueeze(1)).to(F8).to(x.dtype)
        scales.append((top / E4M3_MAX).float().to(x.dtype))
    return codes, torch.stack(scales, 1)
