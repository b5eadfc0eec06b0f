"""CPU reference of the dense operators (8-bit linear, gated half, block norm, token log
probabilities) in numpy float64, written from their formulas; nothing here is shared with
the HIP sources.  Quantization follows its definition step by step in float32, so codes and
scales are exact."""
from __future__ import annotations

import numpy as np

BLOCK = 128
AMAX_FLOOR = np.float32(2.0 ** -96)


def e4m3_values() -> np.ndarray:
    """The value of every e4m3 code 0..255 (4 exponent bits with bias 7, 3 mantissa bits, NaN at 127 and 255)."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
        v[c] = np.nan if c & 127 == 127 else (-mag if c >> 7 else mag)
    return v


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]                             # ascending
_MIDDLES = (_POSITIVE[:-1] + _POSITIVE[1:]) / 2       # exact in float64


def e4m3_encode(v: np.ndarray) -> np.ndarray:
    """Codes of v, to the nearest value, ties to the even code (|v| beyond 448 plus half a step is not used)."""
    v = np.asarray(v, np.float64)
    a = np.abs(np.where(np.isnan(v), 0, v))
    lo = np.searchsorted(_MIDDLES, a, side="left")    # a <= middle[lo]
    tie = (lo < 126) & (a == _MIDDLES[np.minimum(lo, 125)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo)
    code = np.where(np.signbit(v), code | 128, code)
    return np.where(np.isnan(v), 127, code).astype(np.uint8)


def _blocks(v: np.ndarray, amax: np.ndarray):
    """Factor and scale of blocks with these largest magnitudes (float32, each operation rounded once)."""
    a = np.where(np.isnan(amax), amax, np.maximum(amax, AMAX_FLOOR)).astype(np.float32)
    with np.errstate(all="ignore"):
        return np.float32(448) / a, a / np.float32(448)


def quantize(x: np.ndarray):
    """x [t, k] float32 -> codes [t, k] uint8, scale [ceil(k / 128), t] float32."""
    x = np.asarray(x, np.float32)
    t, k = x.shape
    kb = -(-k // BLOCK)
    p = np.zeros((t, kb * BLOCK), np.float32)
    p[:, :k] = x
    p = p.reshape(t, kb, BLOCK)
    factor, scale = _blocks(p, np.abs(p).max(axis=2))
    with np.errstate(all="ignore"):
        codes = e4m3_encode((p * factor[:, :, None]).astype(np.float32))
    return codes.reshape(t, kb * BLOCK)[:, :k].copy(), np.ascontiguousarray(scale.T)


def quantize_weight(w: np.ndarray):
    """w [n, k] float32 -> codes [n, k] uint8, scale [ceil(n / 128), ceil(k / 128)] float32."""
    w = np.asarray(w, np.float32)
    n, k = w.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    p = np.zeros((nb * BLOCK, kb * BLOCK), np.float32)
    p[:n, :k] = w
    p = p.reshape(nb, BLOCK, kb, BLOCK)
    factor, scale = _blocks(p, np.abs(p).max(axis=(1, 3)))
    codes = e4m3_encode((p * factor[:, None, :, None]).astype(np.float32))
    return codes.reshape(nb * BLOCK, kb * BLOCK)[:n, :k].copy(), scale


def values_x(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    return _VALUES[codes] * np.repeat(scale.T.astype(np.float64), BLOCK, axis=1)[:, : codes.shape[1]]


def values_w(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    n, k = codes.shape
    return _VALUES[codes] * np.repeat(np.repeat(scale.astype(np.float64), BLOCK, 0)[:n], BLOCK, 1)[:, :k]


def linear(xv: np.ndarray, wv: np.ndarray):
    """(x . W^T, the sums of the products' magnitudes) in float64."""
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def act(g: np.ndarray, name: str) -> np.ndarray:
    g = np.asarray(g, np.float64)
    if name == "silu":
        return g / (1 + np.exp(-g))
    return g / 2 * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


def norm(v, weight, bias, kind, eps):
    """(normed rows, 1 / sqrt(variance + eps) per row) in float64."""
    v = np.asarray(v, np.float64)
    if kind == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    rstd = 1 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    out = v * rstd
    if weight is not None:
        out = out * weight
    if bias is not None:
        out = out + bias
    return out, rstd


def block_norm(x, residual, pre, post, gate, a, b, eps, kind, pre_bias=None, post_bias=None):
    """(y, h, rstd of h, magnitude of the terms of y) in float64; gate broadcastable to x."""
    z = np.asarray(x, np.float64)
    if post is not None:
        z, _ = norm(z, post, post_bias, kind, eps)
    if gate is not None:
        z = z * gate
    r = 0 if residual is None else a * np.asarray(residual, np.float64)
    y = r + b * z
    h, rstd = norm(y, pre, pre_bias, kind, eps)
    return y, h, rstd, np.abs(r) + np.abs(b * z)


def token_logprobs(logits, targets, top, inv_temperature):
    """(logprob, entropy, rank, ids, top logprobs) of float64 logits, rows of -infinity, NaN
    and +infinity by their definitions."""
    logits = np.asarray(logits, np.float64)
    t, v = logits.shape
    lp, ent, rank = np.zeros(t), np.zeros(t), np.zeros(t, np.int32)
    ids, best = np.zeros((t, top), np.int32), np.zeros((t, top))
    for i in range(t):
        x, y = logits[i], int(targets[i])
        valid = 0 <= y < v
        if np.isnan(x).any() or np.isposinf(x).any():
            lp[i], ent[i], rank[i] = np.nan if valid else 0, np.nan, 0
            ids[i], best[i] = -1, np.nan
            continue
        if np.isneginf(x).all():
            logp, p = np.full(v, -np.inf), np.zeros(v)
        else:
            d = (x - x.max()) * inv_temperature
            logp = d - np.log(np.exp(d).sum())
            p = np.exp(logp)
        ent[i] = -(p[p > 0] * logp[p > 0]).sum()
        if valid:
            lp[i] = logp[y]
            rank[i] = 1 + (x > x[y]).sum() + (x[:y] == x[y]).sum()
        order = np.argsort(-x, kind="stable")[:top]
        ids[i], best[i] = order, logp[order]
    return lp, ent, rank, ids, best
