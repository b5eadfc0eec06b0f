"""Refusals of the 8-bit integer linear and the expert operators, at the C ABI and in the Python wrapper (no GPU): every
bad argument is found before any launch."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from token_adaptive_bit_amd import _lib, api   # noqa: E402
from test_dense_validation import D, Recorder   # noqa: E402

L = _lib.LIB
OK, ARG, SHAPE, RANGE, WS, UNSUP = 0, -1, -2, -3, -4, -6
F32, BF16, E4M3, INT8 = 0, 1, 2, 3
FAKE = 0x7F0000000000          # a 256-byte aligned address that is never dereferenced
P = ctypes.c_void_p
f = P(FAKE)
i32, i8, f32, bf = torch.int32, torch.int8, torch.float32, torch.bfloat16


def desc(n, k, gated=0, experts=1):
    d = _lib.MbqInt8Desc()
    return L.mbq_int8_describe(n, k, gated, experts, ctypes.byref(d)), d


@pytest.mark.parametrize("n,k,gated,experts,rbs,kbs", [(1, 1, 0, 1, 1, 1), (17, 129, 0, 3, 2, 2), (130, 300, 1, 5, 18, 3)])
def test_describe(n, k, gated, experts, rbs, kbs):
    st, d = desc(n, k, gated, experts)
    assert st == OK and (d.row_blocks, d.k_blocks, d.experts, d.gated) == (rbs, kbs, experts, gated)
    assert d.expert_stride == rbs * kbs * 2048 and d.scales_offset == experts * d.expert_stride
    assert d.total_bytes == d.scales_offset + (experts * rbs * 64 + 255) // 256 * 256


def test_describe_refuses():
    for n, k, e in ((0, 1, 1), (1, 0, 1), (-5, 8, 1), ((1 << 24) + 1, 8, 1), (8, 1 << 17, 1), (8, 8, 0), (8, 8, 1025), (1 << 19, 1 << 16, 2)):
        assert desc(n, k, 0, e)[0] == SHAPE
    assert desc(8, 8, 2)[0] == ARG and L.mbq_int8_describe(8, 8, 0, 1, None) == ARG
    assert desc(8, (1 << 17) - 1)[0] == OK


def test_pack_refuses():
    _, d = desc(100, 300)
    _, g = desc(100, 300, 1, 4)
    dp, call = ctypes.byref(d), L.mbq_int8_pack
    assert call(None, 0, f, F32, None, f, None, None) == ARG
    assert call(dp, 1, f, F32, None, f, None, None) == ARG and call(ctypes.byref(g), 2, f, F32, None, f, None, None) == ARG
    assert call(dp, 0, None, F32, None, f, None, None) == ARG and call(dp, 0, f, F32, None, None, None, None) == ARG
    assert call(dp, 0, f, E4M3, f, f, None, None) == ARG and call(dp, 0, f, 9, None, f, None, None) == ARG
    assert call(dp, 0, f, INT8, None, f, None, None) == ARG and call(dp, 0, f, BF16, f, f, None, None) == ARG
    assert call(dp, 0, f, F32, None, P(FAKE + 16), None, None) == ARG and call(dp, 0, P(FAKE + 2), F32, None, f, None, None) == ARG
    assert call(dp, 0, f, INT8, P(FAKE + 2), f, None, None) == ARG and call(dp, 0, f, F32, None, f, P(FAKE + 2), None) == ARG
    for field, st in (("abi", UNSUP), ("k_blocks", SHAPE), ("total_bytes", SHAPE), ("expert_stride", SHAPE), ("experts", SHAPE)):
        bad = _lib.MbqInt8Desc.from_buffer_copy(d)
        setattr(bad, field, getattr(bad, field) + 1)
        assert call(ctypes.byref(bad), 0, f, F32, None, f, None, None) == st


def test_quantize_refuses():
    call = lambda t=4, k=300, x=f, xd=BF16, ldx=300, q=f, ldq=300, s=f: L.mbq_int8_quantize(t, k, x, xd, ldx, q, ldq, s, None)
    assert call(xd=INT8) == ARG and call(xd=E4M3) == ARG
    assert call(x=None) == ARG and call(q=None) == ARG and call(s=None) == ARG
    assert call(x=P(FAKE + 1)) == ARG and call(s=P(FAKE + 2)) == ARG
    assert call(t=-1) == SHAPE and call(t=(1 << 21) + 1) == SHAPE and call(k=0) == SHAPE and call(k=1 << 17) == SHAPE
    assert call(ldx=299) == SHAPE and call(ldq=299) == SHAPE
    assert call(t=0, x=None, q=None, s=None) == OK


def run(d, **kw):
    a = dict(t=4, p=4, x_dtype=BF16, y_dtype=BF16, act=0, reserved=0, x=FAKE, x_scale=None, offsets=None, rows=None, y=FAKE,
             workspace=FAKE, ws_bytes=1 << 40, ldx=d.k)
    packed = kw.pop("packed", f)
    a.update(kw)
    args = _lib.MbqInt8Args(**a)
    return L.mbq_int8_linear(ctypes.byref(d), packed, ctypes.byref(args), None)


@pytest.mark.parametrize("gated", [0, 1])
def test_linear_refuses(gated):
    _, d = desc(100, 304, gated)
    _, many = desc(100, 304, gated, 6)
    _, odd = desc(100, 300, gated)
    assert L.mbq_int8_linear(None, f, None, None) == ARG and L.mbq_int8_linear(ctypes.byref(d), f, None, None) == ARG
    assert run(d, x_dtype=E4M3) == ARG and run(d, y_dtype=INT8) == ARG and run(d, y_dtype=7) == ARG and run(d, reserved=1) == ARG
    assert run(d, act=2) == ARG and run(d, act=-1) == ARG and (gated or run(d, act=1) == ARG)
    assert run(d, packed=None) == ARG and run(d, x=None) == ARG and run(d, y=None) == ARG
    assert run(d, packed=P(FAKE + 16)) == ARG and run(d, x=FAKE + 1) == ARG and run(d, y=FAKE + 1) == ARG
    assert run(d, t=-1, p=-1) == SHAPE and run(d, t=(1 << 21) + 1, p=(1 << 21) + 1) == SHAPE and run(d, ldx=303) == SHAPE
    assert run(d, p=5) == SHAPE                                           # rows of y without rows of x
    assert run(d, rows=FAKE) == ARG                                       # rows without offsets
    assert run(many) == UNSUP                                             # experts without offsets
    assert run(many, offsets=FAKE + 2) == ARG and run(many, offsets=FAKE, rows=FAKE + 1, p=9) == ARG
    assert run(many, offsets=FAKE, rows=FAKE, p=(1 << 24) + 1) == SHAPE and run(many, offsets=FAKE, rows=FAKE, t=0, p=3) == SHAPE
    assert run(many, offsets=FAKE, p=3) == SHAPE
    assert run(d, x_scale=FAKE) == ARG and run(d, x_dtype=INT8) == ARG
    assert run(d, x_dtype=INT8, x_scale=FAKE, x=FAKE + 8) == ARG and run(d, x_dtype=INT8, x_scale=FAKE, ldx=312) == SHAPE
    assert run(d, x_dtype=INT8, x_scale=FAKE + 1) == ARG
    n = ctypes.c_size_t(0)
    size = lambda e, t, p, grouped, xd: L.mbq_int8_workspace(ctypes.byref(e), t, p, grouped, xd, ctypes.byref(n))
    assert size(odd, 4, 4, 0, INT8) == OK and n.value >= 4 * 384            # the codes' copy
    assert run(odd, x_dtype=INT8, x_scale=FAKE, ldx=301, x=FAKE + 1, ws_bytes=n.value - 1) == WS
    assert size(d, 300, 300, 0, BF16) == OK and n.value >= 300 * 388
    for ws, wsb in ((None, 0), (FAKE, n.value - 1), (FAKE + 16, n.value)):
        assert run(d, t=300, p=300, workspace=ws, ws_bytes=wsb) == WS
    assert size(d, 0, 0, 0, BF16) == OK and n.value == 0
    assert size(d, 4, 5, 0, BF16) == SHAPE and size(many, 4, 4, 0, BF16) == SHAPE and size(d, -1, -1, 0, BF16) == SHAPE
    assert size(d, 4, 4, 0, E4M3) == ARG and size(d, 4, 4, 2, BF16) == ARG
    assert L.mbq_int8_workspace(ctypes.byref(d), 4, 4, 0, BF16, None) == ARG
    assert run(d, t=0, p=0, x=None, y=None, packed=None, workspace=None, ws_bytes=0) == OK


def test_route_refuses():
    def call(t=100, e=8, z=f, dt=F32, ld=8, top=2, score=0, norm=1, scale=1.0, ids=f, w=f, perm=f, off=f, place=f, ws=f, wsb=1 << 30):
        return L.mbq_expert_route(t, e, z, dt, ld, top, score, norm, scale, ids, w, perm, off, place, ws, wsb, None)
    assert call(dt=E4M3) == ARG and call(score=2) == ARG and call(norm=2) == ARG
    assert call(t=-1) == SHAPE and call(t=(1 << 21) + 1) == SHAPE and call(e=0) == SHAPE and call(e=1025, ld=1025) == SHAPE
    assert call(top=0) == SHAPE and call(top=9) == SHAPE and call(e=64, ld=64, top=33) == SHAPE and call(ld=7) == SHAPE
    assert call(scale=float("nan")) == RANGE and call(scale=float("inf")) == RANGE
    for name in ("z", "ids", "w", "perm", "off", "place"):
        assert call(**{name: None}) == ARG and call(**{name: P(FAKE + 1)}) == ARG
    n = ctypes.c_size_t(0)
    assert L.mbq_expert_route_workspace(100, 8, ctypes.byref(n)) == OK and n.value > 0
    assert call(ws=None) == WS and call(wsb=n.value - 1) == WS and call(ws=P(FAKE + 4)) == WS
    assert L.mbq_expert_route_workspace(32, 8, ctypes.byref(n)) == OK and n.value == 0
    assert L.mbq_expert_route_workspace(-1, 8, ctypes.byref(n)) == SHAPE and L.mbq_expert_route_workspace(4, 0, ctypes.byref(n)) == SHAPE
    assert L.mbq_expert_route_workspace(4, 8, None) == ARG
    for t in (1, 64, 65, 4096, 4097, 1 << 21):
        for e in (1, 3, 1024):
            assert L.mbq_expert_route_workspace(t, e, ctypes.byref(n)) == OK


def test_combine_refuses():
    def call(t=4, n=100, top=2, p=8, rows=f, dt=BF16, ldr=100, w=f, place=f, res=None, rd=BF16, ldres=100, y=f, ldy=100):
        return L.mbq_expert_combine(t, n, top, p, rows, dt, ldr, w, place, res, rd, ldres, y, ldy, None)
    assert call(dt=INT8) == ARG and call(rd=E4M3) == ARG
    assert call(t=-1) == SHAPE and call(n=0) == SHAPE and call(top=0) == SHAPE and call(top=33) == SHAPE and call(p=-1) == SHAPE
    assert call(p=(1 << 24) + 1) == SHAPE
    for name in ("rows", "w", "place", "y"):
        assert call(**{name: None}) == ARG and call(**{name: P(FAKE + 1)}) == ARG
    assert call(res=P(FAKE + 1)) == ARG
    assert call(ldr=99) == SHAPE and call(ldy=99) == SHAPE and call(res=P(FAKE + 512), ldres=99) == SHAPE and call(res=f, ldres=120) == SHAPE
    assert call(t=0, rows=None, w=None, place=None, y=None) == OK


# --- the Python wrapper: the library's compute calls replaced by a recorder

class Calls(Recorder):
    COMPUTE = {"mbq_int8_pack", "mbq_int8_quantize", "mbq_int8_linear", "mbq_expert_route", "mbq_expert_combine"}


@pytest.fixture
def rec(monkeypatch):
    r = Calls(L)
    monkeypatch.setattr(_lib, "LIB", r)
    monkeypatch.setattr(api, "_stream_of", lambda x: None)
    return r


def z(*shape, dtype=bf):
    return D(torch.zeros(*shape, dtype=dtype))


def packed(n=64, k=256, gated=False, experts=1):
    d = _lib.int8_describe(n, k, gated, experts)
    return api.Int8Linear(d, z(int(d.total_bytes), dtype=torch.uint8))


def refuse(error, text, call):
    with pytest.raises(error, match=text):
        call()


def test_wrapper_refuses(rec):
    p, g, e = packed(), packed(gated=True), packed(experts=4)
    off = z(5, dtype=i32)
    refuse(ValueError, "needs int8_gated", lambda: api.int8_linear(g, z(3, 256)))
    refuse(ValueError, "needs int8_linear", lambda: api.int8_gated(p, z(3, 256)))
    refuse(ValueError, "needs expert_linear", lambda: api.expert_gated(e, z(3, 256), off))
    refuse(ValueError, "several experts", lambda: api.int8_linear(e, z(3, 256)))
    refuse(ValueError, "act must be", lambda: api.int8_gated(g, z(3, 256), act="relu"))
    refuse(ValueError, "has 255 inputs", lambda: api.int8_linear(p, z(3, 255), y=z(3, 64)))
    refuse(TypeError, "scale belongs", lambda: api.int8_linear(p, z(3, 256), scale=z(3, dtype=f32), y=z(3, 64)))
    refuse(TypeError, "scale must be", lambda: api.int8_linear(p, z(3, 256, dtype=i8), y=z(3, 64)))
    refuse(ValueError, "scale has shape", lambda: api.int8_linear(p, z(3, 256, dtype=i8), z(4, dtype=f32), y=z(3, 64)))
    refuse(ValueError, "y has shape", lambda: api.int8_linear(p, z(3, 256), y=z(4, 64)))
    refuse(TypeError, "x has dtype", lambda: api.int8_linear(p, z(3, 256, dtype=torch.float16)))
    refuse(ValueError, "contiguous uint8", lambda: api.int8_linear(api.Int8Linear(p.desc, z(64, dtype=torch.uint8)), z(3, 256), y=z(3, 64)))
    refuse(TypeError, "offsets must be a tensor", lambda: api.expert_linear(e, z(3, 256), None))
    refuse(ValueError, "offsets has shape", lambda: api.expert_linear(e, z(3, 256), z(4, dtype=i32), y=z(3, 64)))
    refuse(TypeError, "offsets has dtype", lambda: api.expert_linear(e, z(3, 256), z(5, dtype=torch.int64), y=z(3, 64)))
    refuse(ValueError, "rows must be 1-D", lambda: api.expert_linear(e, z(3, 256), off, z(3, 2, dtype=i32)))
    refuse(TypeError, "rows has dtype", lambda: api.expert_linear(e, z(3, 256), off, z(6, dtype=torch.int64)))
    refuse(ValueError, "y has shape", lambda: api.expert_linear(e, z(3, 256), off, z(6, dtype=i32), y=z(3, 64)))
    refuse(ValueError, "top must lie", lambda: api.expert_route(z(4, 8, dtype=f32), 9))
    refuse(ValueError, "top must lie", lambda: api.expert_route(z(4, 64, dtype=f32), 33))
    refuse(ValueError, "score must be", lambda: api.expert_route(z(4, 8, dtype=f32), 2, score="tanh"))
    refuse(ValueError, "place has shape", lambda: api.expert_combine(z(8, 16), z(4, 2, dtype=f32), z(4, 3, dtype=i32), y=z(4, 16)))
    refuse(TypeError, "weights has dtype", lambda: api.expert_combine(z(8, 16), z(4, 2), z(4, 2, dtype=i32), y=z(4, 16)))
    refuse(ValueError, "residual has shape", lambda: api.expert_combine(z(8, 16), z(4, 2, dtype=f32), z(4, 2, dtype=i32), z(4, 15), y=z(4, 16)))
    refuse(TypeError, "out_dtype", lambda: api.expert_combine(z(8, 16), z(4, 2, dtype=f32), z(4, 2, dtype=i32), z(4, 16), out_dtype=f32))
    refuse(TypeError, "y has dtype", lambda: api.expert_combine(z(8, 16), z(4, 2, dtype=f32), z(4, 2, dtype=i32), z(4, 16), y=z(4, 16, dtype=f32)))
    refuse(TypeError, "2-D", lambda: api.int8_pack(z(3, 4, 5)))
    refuse(TypeError, "3-D", lambda: api.expert_pack(z(4, 5)))
    refuse(TypeError, "needs its scale", lambda: api.int8_pack(z(4, 5, dtype=i8)))
    refuse(TypeError, "needs its scale", lambda: api.int8_pack(z(4, 5), z(4, dtype=f32)))
    refuse(ValueError, "one shape", lambda: api.int8_pack_gated(z(4, 5), z(4, 6)))
    assert rec.calls == []


def test_wrapper_forwards(rec):
    p, e = packed(), packed(experts=4)
    api.int8_linear(p, z(3, 256), y=z(3, 64))
    api.expert_linear(e, z(3, 256), z(5, dtype=i32), z(6, dtype=i32), y=z(6, 64))
    api.expert_combine(z(8, 16), z(4, 2, dtype=f32), z(4, 2, dtype=i32), y=z(4, 16))
    assert rec.calls == ["mbq_int8_linear", "mbq_int8_linear", "mbq_expert_combine"]
