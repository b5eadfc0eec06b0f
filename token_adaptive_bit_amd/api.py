"""PyTorch-facing wrappers over the C ABI (include/mbq.h).

Tensors are plain CUDA (HIP) tensors; each call checks their shapes, dtypes and device
(the C ABI carries pointers, not sizes, so a mismatch would otherwise read or write past
an allocation), passes their device pointers and the current stream to libmbq and returns
without synchronizing.  No arithmetic happens here.
"""
from __future__ import annotations

import ctypes
import warnings
from dataclasses import dataclass
from typing import NamedTuple

import torch

from . import _lib
from ._lib import (MBQ_BF16, MBQ_E4M3, MBQ_F32, MBQ_MUL_AUTO, MBQ_MUL_BF16, MBQ_MUL_FP8_FP4, MBQ_PATH_AUTO,
                   MBQ_PATH_GENERIC, MbqDesc, MbqError, MbqFp8Desc, MbqOpts, check, describe,
                   fp8_describe)

try:
    from . import _bind  # after _lib: the library and torch's runtime are loaded
except ImportError as e:  # built without torch's headers, or for another torch
    _bind = None
    warnings.warn(f"native binding of the dense operators not loaded ({e}); their calls take the slower way through "
                  "ctypes", RuntimeWarning, stacklevel=2)

__all__ = ["PackedLinear", "pack", "pack_bitplane", "pack_concat", "route", "route_from_logits", "regroup", "linear",
           "linear_workspace", "describe", "MbqError", "MlpRouter", "route_mlp",
           "route_mlp_from_scores", "route_mlp_workspace", "linear_lowrank",
           "linear_lowrank_workspace", "route_linear", "route_linear_workspace", "linear_static", "opts",
           "route_prepare", "route_prepare_workspace", "route_linear_prepared",
           "Fp8Linear", "fp8_describe", "fp8_pack", "fp8_pack_gated", "fp8_quantize", "fp8_linear", "fp8_gated",
           "fp8_linear_workspace", "block_norm", "TokenLogprobs", "token_logprobs", "token_logprobs_workspace"]

_FLOATS = (torch.float32, torch.bfloat16)


def _stream() -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MBQ_F32
    if t.dtype == torch.bfloat16:
        return MBQ_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; expected float32 or bfloat16")


def _p(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _dev(t: torch.Tensor, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _arg(t, name: str, shape, dtypes, device) -> None:
    """A tensor argument: on `device`, contiguous, of this shape and one of these dtypes."""
    _dev(t, name)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")


def _opt(t, name, shape, dtypes, device) -> None:
    if t is not None:
        _arg(t, name, shape, dtypes, device)


def _workspace(ws, name, need, device) -> None:
    if ws is None:
        return
    _dev(ws, name)
    if ws.device != device:
        raise ValueError(f"{name} is on {ws.device}, expected {device}")
    if ws.dtype != torch.uint8 or ws.dim() != 1:
        raise TypeError(f"{name} must be a 1-D uint8 tensor")
    if ws.numel() < need:
        raise ValueError(f"{name} holds {ws.numel()} bytes, the call needs {need}")


_PATHS = {None: MBQ_PATH_AUTO, "auto": MBQ_PATH_AUTO, "generic": MBQ_PATH_GENERIC}
_MULS = {None: MBQ_MUL_AUTO, "auto": MBQ_MUL_AUTO, "bf16": MBQ_MUL_BF16, "fp8fp4": MBQ_MUL_FP8_FP4}


def opts(path: str | None = None, decode_mul: str | None = None, prefill_slots: int = 0,
         decode_launches: int = 0) -> MbqOpts:
    """Kernel choices (mbq_opts): path 'auto' | 'generic'; decode_mul 'auto' | 'bf16' |
    'fp8fp4' (the routed decode step's multiply); prefill_slots, the workgroups the MFMA
    prefill's tile plan assumes run at once (0: the device's compute units);
    decode_launches 0 (the plan's choice), 1 or 2 for the fp8 x fp4 decode step."""
    if path not in _PATHS:
        raise ValueError(f"path must be one of {sorted(k for k in _PATHS if k)}")
    if decode_mul not in _MULS:
        raise ValueError(f"decode_mul must be one of {sorted(k for k in _MULS if k)}")
    if int(prefill_slots) < 0:
        raise ValueError("prefill_slots must be >= 0")
    if int(decode_launches) not in (0, 1, 2):
        raise ValueError("decode_launches must be 0, 1 or 2")
    return MbqOpts(_PATHS[path], _MULS[decode_mul], int(prefill_slots), int(decode_launches))


def _optp(o: MbqOpts | None):
    return None if o is None else ctypes.byref(o)


@dataclass
class PackedLinear:
    """One packed weight: geometry plus the slice-major blob (uint8 device tensor)."""
    desc: MbqDesc
    blob: torch.Tensor

    @property
    def n(self): return self.desc.n

    @property
    def k(self): return self.desc.k

    @property
    def group(self): return self.desc.group

    @property
    def slices(self): return self.desc.slices

    def slice_bytes(self) -> int:
        return int(self.desc.slice_stride)


def _blob(p: PackedLinear, device) -> None:
    _dev(p.blob, "packed blob")
    if p.blob.device != device:
        raise ValueError(f"packed blob is on {p.blob.device}, expected {device}")
    if p.blob.dtype != torch.uint8 or p.blob.numel() < p.desc.total_bytes:
        raise ValueError("packed blob must be uint8 holding at least desc.total_bytes")


def _pack_args(w, status, out, d):
    _dev(w, "w")
    if w.dim() != 2 or w.dtype not in _FLOATS:
        raise TypeError("w must be a 2-D float32 or bfloat16 tensor")
    _opt(status, "status", (1,), (torch.int32,), w.device)
    if out is None:
        out = torch.empty(int(d.total_bytes), dtype=torch.uint8, device=w.device)
    _workspace(out, "out", int(d.total_bytes), w.device)
    return out


def pack(w: torch.Tensor, group: int = 128, slices: int = 3, status: torch.Tensor | None = None,
         out: torch.Tensor | None = None) -> PackedLinear:
    """MoBiSlice pack of W [n, k] (float32 or bfloat16) into a new or given blob."""
    _dev(w, "w")
    n, k = w.shape
    d = describe(n, k, group, slices)
    out = _pack_args(w, status, out, d)
    check(_lib.LIB.mbq_pack(ctypes.byref(d), _p(w), _dtype(w), _p(out), _p(status), _stream()),
          "mbq_pack")
    return PackedLinear(d, out)


def pack_bitplane(w: torch.Tensor, group: int = 128, slices: int = 3,
                  status: torch.Tensor | None = None, out: torch.Tensor | None = None) -> PackedLinear:
    """Bit-plane pack of W [n, k]: slice j is the j-th 2-bit plane of one uniform 2S-bit
    code; the routed linear reads it like any other blob."""
    _dev(w, "w")
    n, k = w.shape
    d = describe(n, k, group, slices)
    out = _pack_args(w, status, out, d)
    check(_lib.LIB.mbq_pack_bitplane(ctypes.byref(d), _p(w), _dtype(w), _p(out), _p(status), _stream()),
          "mbq_pack_bitplane")
    return PackedLinear(d, out)


def pack_concat(ws, group: int = 128, slices: int = 3, status: torch.Tensor | None = None):
    """One blob for weights that read the same activations: W_i [n_i, k] packed as the row
    concatenation (every n_i but the last a multiple of 16).  Returns the PackedLinear and
    the first output column of each weight in the fused output."""
    for i, w in enumerate(ws):
        _dev(w, f"w[{i}]")
        if w.dim() != 2 or w.dtype not in _FLOATS:
            raise TypeError("every weight must be a 2-D float32 or bfloat16 tensor")
        if w.device != ws[0].device:
            raise ValueError("all weights must be on one device")
    k = ws[0].shape[1]
    n = sum(w.shape[0] for w in ws)
    d = describe(n, k, group, slices)
    _opt(status, "status", (1,), (torch.int32,), ws[0].device)
    out = torch.empty(int(d.total_bytes), dtype=torch.uint8, device=ws[0].device)
    starts, row0 = [], 0
    for w in ws:
        if w.shape[1] != k:
            raise ValueError("all weights must have the same number of inputs")
        check(_lib.LIB.mbq_pack_rows(ctypes.byref(d), row0, w.shape[0], _p(w), _dtype(w), _p(out),
                                     _p(status), _stream()), "mbq_pack_rows")
        starts.append(row0)
        row0 += w.shape[0]
    return PackedLinear(d, out), starts


def _route_outputs(t, s, dev, logits, budget, perm, offsets):
    _opt(logits, "logits", (t, s), (torch.float32,), dev)
    _opt(budget, "budget", (t,), (torch.int32,), dev)
    _opt(perm, "perm", (t,), (torch.int32,), dev)
    _opt(offsets, "offsets", (s + 1,), (torch.int32,), dev)
    logits = torch.empty((t, s), dtype=torch.float32, device=dev) if logits is None else logits
    budget = torch.empty(t, dtype=torch.int32, device=dev) if budget is None else budget
    perm = torch.empty(t, dtype=torch.int32, device=dev) if perm is None else perm
    offsets = torch.empty(s + 1, dtype=torch.int32, device=dev) if offsets is None else offsets
    return logits, budget, perm, offsets


def route(x: torch.Tensor, wr: torch.Tensor, logits=None, budget=None, perm=None, offsets=None):
    """Router logits x . wr (float32), budgets 1 + first argmax, stable regroup."""
    _dev(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [t, k]")
    t, k = x.shape
    _dev(wr, "wr")
    if wr.dim() != 2:
        raise ValueError("wr must be 2-D [k, s]")
    s = wr.shape[1]
    _arg(x, "x", (t, k), _FLOATS, x.device)
    _arg(wr, "wr", (k, s), (torch.float32,), x.device)
    logits, budget, perm, offsets = _route_outputs(t, s, x.device, logits, budget, perm, offsets)
    check(_lib.LIB.mbq_route(t, k, s, _p(x), _dtype(x), _p(wr), _p(logits), _p(budget), _p(perm),
                             _p(offsets), _stream()), "mbq_route")
    return logits, budget, perm, offsets


def route_from_logits(logits: torch.Tensor):
    """Route from given float32 logits [t, s] (the bit-exact route contract)."""
    _dev(logits, "logits")
    if logits.dim() != 2 or logits.dtype != torch.float32:
        raise TypeError("logits must be a 2-D float32 tensor")
    t, s = logits.shape
    _, budget, perm, offsets = _route_outputs(t, s, logits.device, None, None, None, None)
    check(_lib.LIB.mbq_route(t, 0, s, None, MBQ_F32, None, _p(logits), _p(budget), _p(perm),
                             _p(offsets), _stream()), "mbq_route")
    return budget, perm, offsets


def regroup(budget: torch.Tensor, slices: int, perm=None, offsets=None):
    """Stable regroup of tokens with given budgets (int32 [t], values in 1..slices)."""
    _dev(budget, "budget")
    if budget.dim() != 1 or budget.dtype != torch.int32:
        raise TypeError("budget must be a 1-D int32 tensor")
    t = budget.shape[0]
    dev = budget.device
    _opt(perm, "perm", (t,), (torch.int32,), dev)
    _opt(offsets, "offsets", (slices + 1,), (torch.int32,), dev)
    perm = torch.empty(t, dtype=torch.int32, device=dev) if perm is None else perm
    offsets = torch.empty(slices + 1, dtype=torch.int32, device=dev) if offsets is None else offsets
    check(_lib.LIB.mbq_regroup(t, slices, _p(budget), _p(perm), _p(offsets), _stream()),
          "mbq_regroup")
    return perm, offsets


@dataclass
class MlpRouter:
    """Weights of the 2-layer MLP router on the device.

    w1 [hidden, k] bfloat16, b1 [hidden] float32, w2 [hidden, slices - 1] float32,
    b2 [slices - 1] float32.
    """
    w1: torch.Tensor
    b1: torch.Tensor
    w2: torch.Tensor
    b2: torch.Tensor

    @property
    def hidden(self): return self.w1.shape[0]

    @property
    def k(self): return self.w1.shape[1]

    @property
    def slices(self): return self.w2.shape[1] + 1


def route_mlp_workspace(t: int, k: int, hidden: int) -> int:
    return _lib.route_mlp_workspace_bytes(t, k, hidden)


def _mlp_outputs(t, s, dev, scores, budget, perm, offsets):
    _opt(scores, "scores", (t, s - 1), (torch.float32,), dev)
    _opt(budget, "budget", (t,), (torch.int32,), dev)
    _opt(perm, "perm", (t,), (torch.int32,), dev)
    _opt(offsets, "offsets", (s + 1,), (torch.int32,), dev)
    scores = torch.empty((t, s - 1), dtype=torch.float32, device=dev) if scores is None else scores
    budget = torch.empty(t, dtype=torch.int32, device=dev) if budget is None else budget
    perm = torch.empty(t, dtype=torch.int32, device=dev) if perm is None else perm
    offsets = torch.empty(s + 1, dtype=torch.int32, device=dev) if offsets is None else offsets
    return scores, budget, perm, offsets


def route_mlp(x: torch.Tensor, r: MlpRouter, delta: float, scores=None, budget=None, perm=None,
              offsets=None, workspace: torch.Tensor | None = None):
    """MLP router scores, threshold-delta budgets and the stable regroup."""
    _dev(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [t, k]")
    t, k = x.shape
    dev = x.device
    _arg(x, "x", (t, k), _FLOATS, dev)
    h = r.w1.shape[0]
    s = r.slices
    _arg(r.w1, "w1", (h, k), (torch.bfloat16,), dev)
    _arg(r.b1, "b1", (h,), (torch.float32,), dev)
    _arg(r.w2, "w2", (h, s - 1), (torch.float32,), dev)
    _arg(r.b2, "b2", (s - 1,), (torch.float32,), dev)
    scores, budget, perm, offsets = _mlp_outputs(t, s, dev, scores, budget, perm, offsets)
    need = route_mlp_workspace(t, k, h)
    _workspace(workspace, "workspace", need, dev)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel()
    check(_lib.LIB.mbq_route_mlp(t, k, s, h, _p(x), _dtype(x), _p(r.w1), _p(r.b1),
                                 _p(r.w2), _p(r.b2), float(delta), _p(scores), _p(budget),
                                 _p(perm), _p(offsets), _p(workspace), ws_bytes, _stream()),
          "mbq_route_mlp")
    return scores, budget, perm, offsets


def route_mlp_from_scores(scores: torch.Tensor, delta: float, budget=None, perm=None,
                          offsets=None):
    """Threshold-delta budgets and regroup from given float32 scores [t, slices - 1]."""
    _dev(scores, "scores")
    if scores.dim() != 2 or scores.dtype != torch.float32:
        raise TypeError("scores must be a 2-D float32 tensor")
    t, r = scores.shape
    s = r + 1
    _, budget, perm, offsets = _mlp_outputs(t, s, scores.device, scores, budget, perm, offsets)
    check(_lib.LIB.mbq_route_mlp(t, 0, s, 0, None, MBQ_F32, None, None, None, None, float(delta),
                                 _p(scores), _p(budget), _p(perm), _p(offsets), None, 0,
                                 _stream()), "mbq_route_mlp")
    return budget, perm, offsets


def linear_workspace(p: PackedLinear, t: int, x_dtype=torch.bfloat16) -> int:
    return _lib.workspace_bytes(p.desc, t, MBQ_BF16 if x_dtype == torch.bfloat16 else MBQ_F32)


def _linear_args(p, x, perm, offsets, out_dtype, y):
    """Checks the routed linear's tensors; returns (t, y)."""
    _dev(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [t, k]")
    t = x.shape[0]
    dev = x.device
    _blob(p, dev)
    _arg(x, "x", (t, p.k), _FLOATS, dev)
    _arg(perm, "perm", (t,), (torch.int32,), dev)
    _arg(offsets, "offsets", (p.slices + 1,), (torch.int32,), dev)
    out_dtype = out_dtype or x.dtype
    if y is None:
        y = torch.empty((t, p.n), dtype=out_dtype, device=dev)
    _arg(y, "y", (t, p.n), _FLOATS, dev)
    return t, y


def linear(p: PackedLinear, x: torch.Tensor, perm: torch.Tensor, offsets: torch.Tensor,
           out_dtype: torch.dtype | None = None, y: torch.Tensor | None = None,
           workspace: torch.Tensor | None = None, options: MbqOpts | None = None) -> torch.Tensor:
    """Routed linear y = x . W^(b(t))^T, original token order."""
    t, y = _linear_args(p, x, perm, offsets, out_dtype, y)
    need = linear_workspace(p, t, x.dtype)
    _workspace(workspace, "workspace", need, x.device)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel()
    check(_lib.LIB.mbq_linear(ctypes.byref(p.desc), _p(p.blob), t, _p(x), _dtype(x), _p(perm),
                              _p(offsets), _p(y), _dtype(y), _p(workspace), ws_bytes, _optp(options),
                              _stream()), "mbq_linear")
    return y


def linear_static(p: PackedLinear, x: torch.Tensor, perm: torch.Tensor, offsets: torch.Tensor,
                  out_dtype: torch.dtype | None = None, y: torch.Tensor | None = None,
                  options: MbqOpts | None = None) -> torch.Tensor:
    """The routed linear without a workspace (mbq_linear_static): for callers that cannot
    allocate; y must then be given.  Calls that overlap on one GPU race (one shared buffer)."""
    t, y = _linear_args(p, x, perm, offsets, out_dtype, y)
    check(_lib.LIB.mbq_linear_static(ctypes.byref(p.desc), _p(p.blob), t, _p(x), _dtype(x), _p(perm),
                                     _p(offsets), _p(y), _dtype(y), _optp(options), _stream()),
          "mbq_linear_static")
    return y


def route_linear_workspace(p: PackedLinear, t: int, x_dtype=torch.bfloat16) -> int:
    return _lib.route_linear_workspace_bytes(p.desc, t, MBQ_BF16 if x_dtype == torch.bfloat16 else MBQ_F32)


def route_prepare_workspace(p: PackedLinear, t: int) -> int:
    n = ctypes.c_size_t(0)
    check(_lib.LIB.mbq_route_prepare_workspace(ctypes.byref(p.desc), t, ctypes.byref(n)),
          "mbq_route_prepare_workspace")
    return int(n.value)


def route_prepare(p: PackedLinear, x: torch.Tensor, wr: torch.Tensor, prep: torch.Tensor | None = None):
    """First launch of the fp8 x fp4 decode step: prepared operands and partial logits of
    x [t, k] (bfloat16, t <= 16) for weights shaped like p.  Returns the prepared buffer."""
    _dev(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [t, k]")
    t = x.shape[0]
    _arg(x, "x", (t, p.k), (torch.bfloat16,), x.device)
    _arg(wr, "wr", (p.k, p.slices), (torch.float32,), x.device)
    need = route_prepare_workspace(p, t)
    if prep is None:
        prep = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _workspace(prep, "prep", need, x.device)
    check(_lib.LIB.mbq_route_prepare(ctypes.byref(p.desc), t, _p(x), _p(wr), _p(prep), prep.numel(), _stream()),
          "mbq_route_prepare")
    return prep


def route_linear_prepared(p: PackedLinear, t: int, prep: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                          y: torch.Tensor | None = None, logits=None, budget=None, perm=None, offsets=None):
    """Second launch: routing from the prepared partial logits and the routed linear on the
    prepared operands.  Returns (y, logits, budget, perm, offsets)."""
    dev = prep.device
    _blob(p, dev)
    _workspace(prep, "prep", route_prepare_workspace(p, t), dev)
    if y is None:
        y = torch.empty((t, p.n), dtype=out_dtype, device=dev)
    _arg(y, "y", (t, p.n), _FLOATS, dev)
    logits, budget, perm, offsets = _route_outputs(t, p.slices, dev, logits, budget, perm, offsets)
    check(_lib.LIB.mbq_route_linear_prepared(ctypes.byref(p.desc), _p(p.blob), t, _p(prep), prep.numel(),
                                             _p(logits), _p(budget), _p(perm), _p(offsets), _p(y), _dtype(y),
                                             _stream()), "mbq_route_linear_prepared")
    return y, logits, budget, perm, offsets


def route_linear(p: PackedLinear, x: torch.Tensor, wr: torch.Tensor, out_dtype: torch.dtype | None = None,
                 y: torch.Tensor | None = None, logits=None, budget=None, perm=None, offsets=None,
                 workspace: torch.Tensor | None = None, options: MbqOpts | None = None):
    """One decode step: route (logits x . wr, budgets, stable regroup) and the routed linear.
    Returns (y, logits, budget, perm, offsets).  For bfloat16 x, t <= 16 and K within one
    workgroup: one launch up to 8 tokens, two from 9 (the fp8 operands prepared once in the
    workspace); otherwise route, then linear."""
    _dev(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [t, k]")
    t = x.shape[0]
    s = p.slices
    dev = x.device
    _blob(p, dev)
    _arg(x, "x", (t, p.k), _FLOATS, dev)
    _arg(wr, "wr", (p.k, s), (torch.float32,), dev)
    out_dtype = out_dtype or x.dtype
    if y is None:
        y = torch.empty((t, p.n), dtype=out_dtype, device=dev)
    _arg(y, "y", (t, p.n), _FLOATS, dev)
    logits, budget, perm, offsets = _route_outputs(t, s, dev, logits, budget, perm, offsets)
    need = route_linear_workspace(p, t, x.dtype)
    _workspace(workspace, "workspace", need, dev)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel()
    check(_lib.LIB.mbq_route_linear(ctypes.byref(p.desc), _p(p.blob), t, _p(x), _dtype(x), _p(wr),
                                    _p(logits), _p(budget), _p(perm), _p(offsets), _p(y), _dtype(y),
                                    _p(workspace), ws_bytes, _optp(options), _stream()),
          "mbq_route_linear")
    return y, logits, budget, perm, offsets


def linear_lowrank_workspace(p: PackedLinear, t: int, rank: int, x_dtype=torch.bfloat16) -> int:
    return _lib.lowrank_workspace_bytes(p.desc, t, MBQ_BF16 if x_dtype == torch.bfloat16 else MBQ_F32,
                                        rank)


def linear_lowrank(p: PackedLinear, x: torch.Tensor, perm: torch.Tensor, offsets: torch.Tensor,
                   a: torch.Tensor, b: torch.Tensor, out_dtype: torch.dtype | None = None,
                   y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   options: MbqOpts | None = None) -> torch.Tensor:
    """Routed linear plus the low-rank side path: y = x . W^(b(t))^T + (x . a^T) . b^T,
    a [rank, k] and b [n, rank] bfloat16."""
    t, y = _linear_args(p, x, perm, offsets, out_dtype, y)
    _dev(a, "a")
    if a.dim() != 2:
        raise ValueError("a must be 2-D [rank, k]")
    rank = a.shape[0]
    _arg(a, "a", (rank, p.k), (torch.bfloat16,), x.device)
    _arg(b, "b", (p.n, rank), (torch.bfloat16,), x.device)
    need = linear_lowrank_workspace(p, t, rank, x.dtype)
    _workspace(workspace, "workspace", need, x.device)
    if need and workspace is None:  # zero-filled: the call state starts from zero
        workspace = torch.zeros(need, dtype=torch.uint8, device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel()
    check(_lib.LIB.mbq_linear_lowrank(ctypes.byref(p.desc), _p(p.blob), t, _p(x), _dtype(x), _p(perm),
                                      _p(offsets), _p(a), _p(b), rank, _p(y), _dtype(y), _p(workspace),
                                      ws_bytes, _optp(options), _stream()), "mbq_linear_lowrank")
    return y


# --- dense operators: the 8-bit linear, its gated form, the norms around a block and the
# --- log probabilities of tokens.  A decode step makes many of these calls and each runs for
# --- a few microseconds, so ordinary calls (plain contiguous tensors, no buffers given) are
# --- checked and made by _bind; what it leaves alone comes back here, where the checks name
# --- what is wrong.  Without _bind every call comes here: the same kernels, a few microseconds later.

_F8 = torch.float8_e4m3fn
_CODE = {torch.float32: MBQ_F32, torch.bfloat16: MBQ_BF16, _F8: MBQ_E4M3}
_F32S, _F8S, _IDS = (torch.float32,), (_F8,), (torch.int32, torch.int64)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream_of(x: torch.Tensor):
    """The current stream of x's device, which has to be the current one."""
    i = x.get_device()
    if i != _current_device():
        raise ValueError(f"x is on cuda:{i}, the current device is cuda:{_current_device()}")
    return _raw_stream(i)


def _bound(x) -> bool:
    return _bind is not None and type(x) is torch.Tensor and x.is_cuda


def _rows(t, name: str, dtypes, dev=None, shape=None) -> int:
    """A 2-D tensor whose rows may lie apart but are contiguous inside; returns the row stride."""
    if type(t) is torch.Tensor and t.is_cuda and t.dim() == 2 and t.dtype in dtypes and t.is_contiguous() \
            and (dev is None or t.get_device() == dev) and (shape is None or t.shape == shape):
        return t.shape[1]
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{name} has overlapping rows")
    return ld


def _flat(t, name: str, dtypes, dev, shape) -> int:
    """A contiguous tensor of this shape; returns its address."""
    if not (type(t) is torch.Tensor and t.is_cuda and t.shape == shape and t.dtype in dtypes and t.get_device() == dev
            and t.is_contiguous()):
        _dev(t, name)
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.dtype not in dtypes:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    return t.data_ptr()


def _scratch(ws, need: int, x: torch.Tensor):
    """The workspace given, or a new one; returns (tensor to keep until the call, address, bytes)."""
    if ws is None:
        if not need:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    else:
        _workspace(ws, "workspace", need, x.device)
    return ws, ws.data_ptr(), ws.numel()


@dataclass
class Fp8Linear:
    """A packed 8-bit weight, or the two of a gated half: geometry plus the blob."""
    desc: MbqFp8Desc
    blob: torch.Tensor

    def __post_init__(self):
        self._sizes = {}

    @property
    def n(self): return self.desc.n

    @property
    def k(self): return self.desc.k

    @property
    def gated(self): return bool(self.desc.gated)

    def _workspace_bytes(self, t: int, code: int) -> int:
        """Sizes already asked for, by tokens and type (they depend on nothing else)."""
        need = self._sizes.get((t, code))
        if need is None:
            need = self._sizes[(t, code)] = _lib.fp8_linear_workspace_bytes(self.desc, t, code)
        return need


def _fp8_pack(ws, scales, status, out) -> Fp8Linear:
    for w, s in zip(ws, scales):
        _dev(w, "w")
        if w.dim() != 2 or w.dtype not in _CODE:
            raise TypeError("w must be a 2-D float32, bfloat16 or float8_e4m3fn tensor")
        if w.shape != ws[0].shape:
            raise ValueError(f"both weights must have one shape, got {tuple(ws[0].shape)} and {tuple(w.shape)}")
        if w.device != ws[0].device:
            raise ValueError("both weights must be on one device")
        if (w.dtype == _F8) != (s is not None):
            raise TypeError("a float8_e4m3fn weight needs its scale, and only that")
        _opt(s, "scale", (-(-w.shape[0] // 128), -(-w.shape[1] // 128)), _F32S, w.device)
    n, k = ws[0].shape
    dev = ws[0].device
    _opt(status, "status", (1,), (torch.int32,), dev)
    d = fp8_describe(n, k, len(ws) == 2)
    if out is None:
        out = torch.empty(int(d.total_bytes), dtype=torch.uint8, device=dev)
    _workspace(out, "out", int(d.total_bytes), dev)
    stream = _stream_of(ws[0])
    for part, (w, s) in enumerate(zip(ws, scales)):
        check(_lib.LIB.mbq_fp8_pack(ctypes.byref(d), part, _p(w), _CODE[w.dtype], _p(s), _p(out), _p(status), stream),
              "mbq_fp8_pack")
    return Fp8Linear(d, out)


def fp8_pack(w: torch.Tensor, scale: torch.Tensor | None = None, status: torch.Tensor | None = None,
             out: torch.Tensor | None = None) -> Fp8Linear:
    """8-bit pack of W [n, k]: float32 or bfloat16 (quantized to e4m3, one scale per 128 x 128
    block), or float8_e4m3fn codes with their scale [ceil(n / 128), ceil(k / 128)] float32."""
    return _fp8_pack((w,), (scale,), status, out)


def fp8_pack_gated(w_gate: torch.Tensor, w_up: torch.Tensor, scale_gate: torch.Tensor | None = None,
                   scale_up: torch.Tensor | None = None, status: torch.Tensor | None = None,
                   out: torch.Tensor | None = None) -> Fp8Linear:
    """The two weights [n, k] of a gated half in one blob, for fp8_gated."""
    return _fp8_pack((w_gate, w_up), (scale_gate, scale_up), status, out)


def fp8_quantize(x: torch.Tensor, q: torch.Tensor | None = None, scale: torch.Tensor | None = None):
    """e4m3 codes of x [t, k] per token and 128 inputs.  Returns (q [t, k] float8_e4m3fn,
    scale [ceil(k / 128), t] float32): x is about q * scale."""
    if q is None and scale is None and _bound(x):
        r = _bind.fp8_quantize(x, dev := _current_device(), _raw_stream(dev))
        if r is not None:
            return r
    ldx = _rows(x, "x", _FLOATS)
    t, k = x.shape
    dev, kb = x.get_device(), -(-k // 128)
    if q is None:
        q = torch.empty_like(x, dtype=_F8)
    ldq = _rows(q, "q", _F8S, dev, (t, k))
    if scale is None:
        scale = torch.empty(kb, t, dtype=torch.float32, device=x.device)
    check(_lib.LIB.mbq_fp8_quantize(t, k, x.data_ptr(), _CODE[x.dtype], ldx, q.data_ptr(), ldq,
                                    _flat(scale, "scale", _F32S, dev, (kb, t)), _stream_of(x)), "mbq_fp8_quantize")
    return q, scale


def fp8_linear_workspace(p: Fp8Linear, t: int, x_dtype=torch.bfloat16) -> int:
    return p._workspace_bytes(t, _CODE[x_dtype])


def _fp8_run(p, x, scale, act, out_dtype, y, workspace):
    if y is None and workspace is None and _bound(x):
        r = _bind.fp8(ctypes.addressof(p.desc), p.blob, x, scale, -1 if act is None else act, out_dtype, dev := _current_device(),
                      _raw_stream(dev))
        if r is not None:
            return r
    ldx = _rows(x, "x", _CODE)
    t, k = x.shape
    dev, code, n, blob = x.get_device(), _CODE[x.dtype], p.desc.n, p.blob
    if k != p.desc.k:
        raise ValueError(f"x has {k} inputs, the weight {p.desc.k}")
    if blob.dtype != torch.uint8 or blob.get_device() != dev or not blob.is_contiguous() or blob.numel() < p.desc.total_bytes:
        raise ValueError(f"packed blob must be contiguous uint8 on cuda:{dev} holding at least desc.total_bytes")
    if code == MBQ_E4M3:
        scale = _flat(scale, "scale", _F32S, dev, (p.desc.k_blocks, t))
    elif scale is not None:
        raise TypeError("scale belongs to float8_e4m3fn activations")
    if y is None:
        y = torch.empty(t, n, dtype=out_dtype or (torch.bfloat16 if code == MBQ_E4M3 else x.dtype), device=x.device)
    y_ptr, y_code = _flat(y, "y", _FLOATS, dev, (t, n)), _CODE[y.dtype]
    _ws, ws_ptr, ws_bytes = _scratch(workspace, p._workspace_bytes(t, code), x)
    if act is None:
        check(_lib.LIB.mbq_fp8_linear(ctypes.byref(p.desc), blob.data_ptr(), t, x.data_ptr(), code, ldx, scale, y_ptr, y_code, ws_ptr,
                                      ws_bytes, _stream_of(x)), "mbq_fp8_linear")
    else:
        check(_lib.LIB.mbq_fp8_gated(ctypes.byref(p.desc), blob.data_ptr(), t, x.data_ptr(), code, ldx, scale, act, y_ptr, y_code,
                                     ws_ptr, ws_bytes, _stream_of(x)), "mbq_fp8_gated")
    return y


def fp8_linear(p: Fp8Linear, x: torch.Tensor, scale: torch.Tensor | None = None,
               out_dtype: torch.dtype | None = None, y: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """8-bit linear y = x . W^T: x [t, k] float32 or bfloat16 (quantized per token and 128
    inputs within the call), or the codes and scale of fp8_quantize / block_norm."""
    if p.desc.gated:
        raise ValueError("a gated blob needs fp8_gated")
    return _fp8_run(p, x, scale, None, out_dtype, y, workspace)


_ACTS = {"silu": _lib.MBQ_ACT_SILU, "gelu_tanh": _lib.MBQ_ACT_GELU_TANH}


def fp8_gated(p: Fp8Linear, x: torch.Tensor, scale: torch.Tensor | None = None, act: str = "silu",
              out_dtype: torch.dtype | None = None, y: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Gated half of a feed-forward block: act(x . Wg^T) * (x . Wu^T) on a gated blob."""
    if not p.desc.gated:
        raise ValueError("fp8_gated needs a blob of fp8_pack_gated")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    return _fp8_run(p, x, scale, _ACTS[act], out_dtype, y, workspace)


_KINDS = {"rms": _lib.MBQ_NORM_RMS, "layer": _lib.MBQ_NORM_LAYER}


def block_norm(x: torch.Tensor, residual: torch.Tensor | None = None, pre: torch.Tensor | None = None,
               post: torch.Tensor | None = None, gate: torch.Tensor | None = None, residual_scale: float = 1.0,
               gate_scale: float = 1.0, eps: float = 1e-6, kind: str = "rms", pre_bias: torch.Tensor | None = None,
               post_bias: torch.Tensor | None = None, quantized: bool = False, out_dtype: torch.dtype | None = None,
               y: torch.Tensor | None = None, h: torch.Tensor | None = None, scale: torch.Tensor | None = None):
    """The norms around a block: y = residual_scale * residual + gate_scale * gate * z with
    z = norm(x; post) if post is given, else x, and h = norm(y; pre).

    x [t, k]; residual [t, k] or None; pre, post, pre_bias, post_bias [k] float32; gate None,
    [k] or [t] float32 (with t == k: per channel), or [t, k] of x's type; kind 'rms' or
    'layer'.  y has residual's type (x's without one) and may be residual itself; h has x's
    type unless out_dtype says another.  Returns (y, h), or with quantized (y, codes [t, k]
    float8_e4m3fn, scale [ceil(k / 128), t] float32), which fp8_linear takes."""
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of {sorted(_KINDS)}")
    if y is None and h is None and scale is None and _bound(x):
        r = _bind.block_norm(x, residual, pre, post, gate, residual_scale, gate_scale, eps, _KINDS[kind], pre_bias,
                             post_bias, quantized, out_dtype, dev := _current_device(), _raw_stream(dev))
        if r is not None:
            return r
    ldx = _rows(x, "x", _FLOATS)
    shape = x.shape
    t, k = shape
    dev = x.get_device()
    r_dtype, r_ptr, ldr = x.dtype, 0, 0
    if residual is not None:
        ldr = _rows(residual, "residual", _FLOATS, dev, shape)
        r_dtype, r_ptr = residual.dtype, residual.data_ptr()
    pre_ptr = 0 if pre is None else _flat(pre, "pre", _F32S, dev, (k,))
    post_ptr = 0 if post is None else _flat(post, "post", _F32S, dev, (k,))
    preb_ptr = 0 if pre_bias is None else _flat(pre_bias, "pre_bias", _F32S, dev, (k,))
    postb_ptr = 0 if post_bias is None else _flat(post_bias, "post_bias", _F32S, dev, (k,))
    gate_kind = gate_ptr = 0
    if gate is not None:
        if not isinstance(gate, torch.Tensor):
            raise TypeError("gate must be a tensor")
        if gate.dim() == 2:
            gate_kind, gate_ptr = _lib.MBQ_GATE_FULL, _flat(gate, "gate", (x.dtype,), dev, shape)
        elif gate.shape == (k,):
            gate_kind, gate_ptr = _lib.MBQ_GATE_CHANNEL, _flat(gate, "gate", _F32S, dev, (k,))
        else:
            gate_kind, gate_ptr = _lib.MBQ_GATE_TOKEN, _flat(gate, "gate", _F32S, dev, (t,))
    if y is None:
        y, ldy = torch.empty_like(x, dtype=r_dtype), k
    else:
        ldy = _rows(y, "y", (r_dtype,), dev, shape)
    if h is None:
        h, ldh = torch.empty_like(x, dtype=_F8 if quantized else out_dtype or x.dtype), k
    else:
        ldh = _rows(h, "h", _F8S if quantized else _FLOATS if out_dtype is None else (out_dtype,), dev, shape)
    s_ptr = 0
    if quantized:
        if scale is None:
            scale = torch.empty(-(-k // 128), t, dtype=torch.float32, device=x.device)
        s_ptr = _flat(scale, "scale", _F32S, dev, (-(-k // 128), t))
    elif scale is not None:
        raise TypeError("scale belongs to quantized=True")
    if h.dtype not in _CODE:
        raise TypeError(f"out_dtype {h.dtype}, expected float32 or bfloat16")
    args = _lib.BLOCK_NORM_ARGS.pack(t, k, _KINDS[kind], gate_kind, _CODE[x.dtype], _CODE[r_dtype], _CODE[h.dtype],
                                     post is not None, x.data_ptr(), r_ptr, post_ptr, postb_ptr, pre_ptr, preb_ptr,
                                     gate_ptr, y.data_ptr(), h.data_ptr(), s_ptr, ldx, ldr, ldy, ldh, residual_scale,
                                     gate_scale, eps)
    check(_lib.LIB.mbq_block_norm(args, _stream_of(x)), "mbq_block_norm")
    return (y, h, scale) if quantized else (y, h)


class TokenLogprobs(NamedTuple):
    """Per row: log probability of the target, entropy (nats), rank of the target (1 is the
    best), and with top > 0 the best tokens and their log probabilities."""
    logprob: torch.Tensor
    entropy: torch.Tensor
    rank: torch.Tensor
    top_ids: torch.Tensor | None = None
    top_logprobs: torch.Tensor | None = None


def token_logprobs_workspace(t: int, v: int, top: int = 0) -> int:
    return _lib.token_logprobs_workspace_bytes(t, v, top)


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, top: int = 0, inv_temperature: float = 1.0,
                   workspace: torch.Tensor | None = None) -> TokenLogprobs:
    """Log probabilities of targets [t] (int32 or int64; outside [0, v): a padded position)
    under softmax(inv_temperature * logits [t, v]), with entropy, rank and the top (<= 64)
    alternatives, equal logits by ascending token."""
    if workspace is None and _bound(logits):
        r = _bind.token_logprobs(logits, targets, top, inv_temperature, dev := _current_device(), _raw_stream(dev))
        if r is not None:
            return TokenLogprobs._make(r)
    ld = _rows(logits, "logits", _FLOATS)
    t, v = logits.shape
    dev = logits.get_device()
    tg_ptr = _flat(targets, "targets", _IDS, dev, (t,))
    if not 0 <= top <= min(v, _lib.MBQ_MAX_TOP):
        raise ValueError(f"top must lie in 0 .. {min(v, _lib.MBQ_MAX_TOP)}")
    device = logits.device
    logprob = torch.empty(t, dtype=torch.float32, device=device)
    entropy = torch.empty_like(logprob)
    rank = torch.empty_like(logprob, dtype=torch.int32)
    ids = best = ids_ptr = best_ptr = None
    if top:
        best = torch.empty(t, top, dtype=torch.float32, device=device)
        ids = torch.empty_like(best, dtype=torch.int32)
        ids_ptr, best_ptr = ids.data_ptr(), best.data_ptr()
    _ws, ws_ptr, ws_bytes = _scratch(workspace, _lib.token_logprobs_workspace_bytes(t, v, top), logits)
    check(_lib.LIB.mbq_token_logprobs(t, v, logits.data_ptr(), _CODE[logits.dtype], ld, tg_ptr,
                                      32 if targets.dtype == torch.int32 else 64, inv_temperature, top,
                                      logprob.data_ptr(), entropy.data_ptr(), rank.data_ptr(), ids_ptr, best_ptr, ws_ptr,
                                      ws_bytes, _stream_of(logits)), "mbq_token_logprobs")
    return TokenLogprobs(logprob, entropy, rank, ids, best)
