"""CPU reference of the 8-bit integer linear and the expert operators in numpy float64, written from their formulas; nothing
here is shared with the HIP sources.  Quantization follows its definition step by step in float32, so codes and scales are
exact, and products of codes are summed as whole numbers."""
from __future__ import annotations

import numpy as np

AMAX_FLOOR = np.float32(2.0 ** -96)


def quantize(x: np.ndarray):
    """x [..., k] float32 -> codes [..., k] int8, scale [...] float32, one per row."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        a = np.maximum(np.abs(x).max(axis=-1), AMAX_FLOOR)
        bad = ~np.isfinite(x).all(axis=-1)
        factor = np.where(bad, np.float32(0), np.float32(127) / a).astype(np.float32)
        scale = np.where(bad, np.float32(np.nan), a / np.float32(127)).astype(np.float32)
        v = (x * factor[..., None]).astype(np.float32)
    codes = np.rint(np.where(bad[..., None], 0, v)).astype(np.int8)   # to nearest, ties to even
    return codes, scale


def product(xq, xs, wq, ws):
    """(x . W^T, the sums as whole numbers): codes and scales of x [t, k] and of a weight [n, k]."""
    acc = xq.astype(np.int64) @ wq.astype(np.int64).T
    return acc * (xs.astype(np.float64)[:, None] * ws.astype(np.float64)[None]), acc


def gate(g, u, name: str):
    """act(g) * u; the tanh form of gelu by (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)), which keeps its digits where tanh nears -1."""
    a = g if name == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-a)) * u


def order(logits):
    """Experts of every token by descending logit, equal ones by ascending index."""
    return np.argsort(-np.asarray(logits, np.float64), axis=1, kind="stable")


def route(logits, top, score="softmax", normalize=True, weight_scale=1.0):
    """(ids, weights float64, perm, offsets, place) of float64 logits."""
    z = np.asarray(logits, np.float64)
    t, e = z.shape
    ids, weights = np.full((t, top), -1, np.int32), np.zeros((t, top))
    for i in range(t):
        if np.isnan(z[i]).any() or np.isposinf(z[i]).any():
            weights[i] = np.nan
            continue
        chosen = [j for j in order(z[i : i + 1])[0][:top] if z[i, j] > -np.inf]
        if not chosen:
            continue
        if score == "softmax":
            p = np.exp(z[i] - z[i].max())
            s = p[chosen] / (p[chosen].sum() if normalize else p.sum())
        else:
            log_s = -np.logaddexp(0, -z[i][chosen])
            s = np.exp(log_s - log_s.max()) if normalize else np.exp(log_s)
            s = s / s.sum() if normalize else s
        ids[i, : len(chosen)] = chosen
        weights[i, : len(chosen)] = s * weight_scale
    return (ids, weights) + group(ids, e)


def group(ids, experts):
    """(perm, offsets, place) of the token copies, by expert and then by token; ids of -1 have no copy."""
    t, top = ids.shape
    perm, place = np.full(t * top, -1, np.int32), np.full((t, top), -1, np.int32)
    offsets, at = np.zeros(experts + 1, np.int32), 0
    for e in range(experts):
        for i, j in zip(*np.nonzero(ids == e)):
            perm[at], place[i, j] = i, at
            at += 1
        offsets[e + 1] = at
    return perm, offsets, place


def combine(rows, weights, place, residual=None):
    """(y, the terms' magnitudes) in float64."""
    rows, weights = np.asarray(rows, np.float64), np.asarray(weights, np.float64)
    t, top = place.shape
    y = np.zeros((t, rows.shape[1])) if residual is None else np.asarray(residual, np.float64).copy()
    mags = np.abs(y)
    for i in range(t):
        for j in range(top):
            row = rows[place[i, j]] if 0 <= place[i, j] < len(rows) else np.zeros(rows.shape[1])
            y[i] += weights[i, j] * row
            mags[i] += np.abs(weights[i, j] * row)
    return y, mags
