"""Refusals of the dense operators, at the C ABI and in the Python binding (no GPU): every
bad argument is found before any launch."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from token_adaptive_bit_amd import _lib, api   # noqa: E402

L = _lib.LIB
OK, ARG, SHAPE, RANGE, WS, UNSUP = 0, -1, -2, -3, -4, -6
F32, BF16, E4M3 = 0, 1, 2
FAKE = 0x7F0000000000          # a 256-byte aligned address that is never dereferenced
P = ctypes.c_void_p
f = P(FAKE)


def desc(n, k, gated=0):
    d = _lib.MbqFp8Desc()
    return L.mbq_fp8_describe(n, k, gated, ctypes.byref(d)), d


@pytest.mark.parametrize("n,k,gated,rbs,kbs,scales", [(1, 1, 0, 1, 1, 1), (16, 128, 0, 1, 1, 1), (17, 129, 0, 2, 2, 2),
                                                      (130, 300, 0, 9, 3, 6), (130, 300, 1, 18, 3, 12),
                                                      (18944, 3584, 0, 1184, 28, 148 * 28)])
def test_describe(n, k, gated, rbs, kbs, scales):
    st, d = desc(n, k, gated)
    assert st == OK and (d.row_blocks, d.k_blocks) == (rbs, kbs)
    assert d.scales_offset == rbs * kbs * 2048
    assert d.total_bytes == d.scales_offset + (scales * 4 + 255) // 256 * 256


def test_describe_refuses():
    for n, k in ((0, 1), (1, 0), (-5, 8), ((1 << 24) + 1, 8), (8, (1 << 24) + 1), (1 << 19, 1 << 17)):
        assert desc(n, k)[0] == SHAPE
    assert desc(8, 8, 2)[0] == ARG and L.mbq_fp8_describe(8, 8, 0, None) == ARG


def test_pack_refuses():
    _, d = desc(100, 300)
    _, g = desc(100, 300, 1)
    dp = ctypes.byref(d)
    call = L.mbq_fp8_pack
    assert call(None, 0, f, F32, None, f, None, None) == ARG
    assert call(dp, 1, f, F32, None, f, None, None) == ARG and call(ctypes.byref(g), 2, f, F32, None, f, None, None) == ARG
    assert call(dp, -1, f, F32, None, f, None, None) == ARG
    assert call(dp, 0, None, F32, None, f, None, None) == ARG and call(dp, 0, f, F32, None, None, None, None) == ARG
    assert call(dp, 0, f, 3, None, f, None, None) == ARG
    assert call(dp, 0, f, E4M3, None, f, None, None) == ARG and call(dp, 0, f, F32, f, f, None, None) == ARG
    assert call(dp, 0, f, F32, None, P(FAKE + 16), None, None) == ARG
    assert call(dp, 0, P(FAKE + 2), F32, None, f, None, None) == ARG
    assert call(dp, 0, P(FAKE + 1), BF16, None, f, None, None) == ARG
    assert call(dp, 0, f, F32, None, f, P(FAKE + 2), None) == ARG
    for field, st in (("abi", UNSUP), ("k_blocks", SHAPE), ("total_bytes", SHAPE)):
        bad = _lib.MbqFp8Desc.from_buffer_copy(d)
        setattr(bad, field, getattr(bad, field) + 1)
        assert call(ctypes.byref(bad), 0, f, F32, None, f, None, None) == st


def test_quantize_refuses():
    call = lambda t=4, k=300, x=f, xd=BF16, ldx=300, q=f, ldq=300, s=f: L.mbq_fp8_quantize(t, k, x, xd, ldx, q, ldq, s, None)
    assert call(xd=E4M3) == ARG and call(xd=9) == ARG
    assert call(x=None) == ARG and call(q=None) == ARG and call(s=None) == ARG
    assert call(x=P(FAKE + 1)) == ARG and call(s=P(FAKE + 2)) == ARG
    assert call(t=-1) == SHAPE and call(t=(1 << 21) + 1) == SHAPE and call(k=0) == SHAPE
    assert call(ldx=299) == SHAPE and call(ldq=299) == SHAPE
    assert call(t=0, x=None, q=None, s=None) == OK


def linear_call(d, gated=False, **kw):
    a = dict(desc=ctypes.byref(d), packed=f, t=4, x=f, xd=BF16, ldx=d.k, xs=None, act=0, y=f, yd=BF16, ws=f, wsb=1 << 40)
    a.update(kw)
    head = (a["desc"], a["packed"], a["t"], a["x"], a["xd"], a["ldx"], a["xs"])
    tail = (a["y"], a["yd"], a["ws"], a["wsb"], None)
    return L.mbq_fp8_gated(*head, a["act"], *tail) if gated else L.mbq_fp8_linear(*head, *tail)


@pytest.mark.parametrize("gated", [False, True])
def test_linear_refuses(gated):
    _, d = desc(100, 304, int(gated))
    _, other = desc(100, 304, int(not gated))
    call = lambda **kw: linear_call(d, gated, **kw)
    assert call(desc=None) == ARG and call(desc=ctypes.byref(other)) == UNSUP
    assert call(xd=3) == ARG and call(yd=E4M3) == ARG and call(yd=7) == ARG
    assert call(packed=None) == ARG and call(x=None) == ARG and call(y=None) == ARG
    assert call(packed=P(FAKE + 16)) == ARG and call(x=P(FAKE + 1)) == ARG and call(y=P(FAKE + 1)) == ARG
    assert call(t=-1) == SHAPE and call(t=(1 << 21) + 1) == SHAPE and call(ldx=303) == SHAPE
    assert call(xs=f) == ARG                                            # scales without codes
    assert call(xd=E4M3) == ARG                                         # codes without scales
    assert call(xd=E4M3, xs=f, x=P(FAKE + 8)) == ARG and call(xd=E4M3, xs=f, ldx=312) == SHAPE
    _, odd = desc(100, 300, int(gated))
    n = ctypes.c_size_t(0)
    # k not a multiple of 16: the codes' copy lives in the workspace
    assert L.mbq_fp8_linear_workspace(ctypes.byref(odd), 4, E4M3, ctypes.byref(n)) == OK and n.value == 4 * 384
    assert linear_call(odd, gated, xd=E4M3, xs=f, ldx=299) == SHAPE
    assert linear_call(odd, gated, xd=E4M3, xs=f, ldx=301, x=P(FAKE + 1), wsb=n.value - 1) == WS
    # 32 tokens: codes and scales live in the workspace
    assert L.mbq_fp8_linear_workspace(ctypes.byref(d), 32, BF16, ctypes.byref(n)) == OK and n.value > 0
    for ws, wsb in ((None, 0), (f, n.value - 1), (P(FAKE + 16), n.value)):
        assert call(t=32, ws=ws, wsb=wsb) == WS
    assert L.mbq_fp8_linear_workspace(ctypes.byref(d), 0, BF16, ctypes.byref(n)) == OK and n.value == 0
    assert L.mbq_fp8_linear_workspace(ctypes.byref(d), -1, BF16, ctypes.byref(n)) == SHAPE
    assert L.mbq_fp8_linear_workspace(ctypes.byref(d), 4, 5, ctypes.byref(n)) == ARG
    assert L.mbq_fp8_linear_workspace(ctypes.byref(d), 4, BF16, None) == ARG
    assert call(t=0, x=None, y=None, packed=None, ws=None, wsb=0) == OK
    if gated:
        assert call(act=2) == ARG and call(act=-1) == ARG


def test_packed_arguments_match_the_struct():
    """The binding packs the arguments of mbq_block_norm itself: every field where the struct has it."""
    a = _lib.MbqBlockNormArgs.from_buffer_copy(_lib.BLOCK_NORM_ARGS.pack(*range(1, 26)))
    got = [getattr(a, name) for name, _ in _lib.MbqBlockNormArgs._fields_]
    assert got == list(range(1, 26)) and _lib.BLOCK_NORM_ARGS.size == ctypes.sizeof(_lib.MbqBlockNormArgs)


def norm_call(**kw):
    a = _lib.MbqBlockNormArgs(t=4, k=100, kind=0, gate_kind=0, x_dtype=BF16, r_dtype=BF16, h_dtype=BF16, post=1, x=FAKE,
                              residual=FAKE, post_weight=FAKE, pre_weight=FAKE, y=FAKE, h=FAKE, ldx=100, ldr=100, ldy=100,
                              ldh=100, residual_scale=1.0, gate_scale=1.0, eps=1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    return L.mbq_block_norm(ctypes.byref(a), None)


def test_block_norm_refuses():
    assert L.mbq_block_norm(None, None) == ARG
    for field in ("x_dtype", "r_dtype", "h_dtype"):
        assert norm_call(**{field: 3}) == ARG
    assert norm_call(x_dtype=E4M3) == ARG and norm_call(r_dtype=E4M3) == ARG
    assert norm_call(kind=2) == ARG and norm_call(gate_kind=4) == ARG and norm_call(gate_kind=-1) == ARG and norm_call(post=2) == ARG
    assert norm_call(t=-1) == SHAPE and norm_call(t=(1 << 21) + 1) == SHAPE and norm_call(k=0) == SHAPE
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert norm_call(eps=eps) == RANGE
    assert norm_call(gate_scale=float("nan")) == RANGE and norm_call(residual_scale=float("inf")) == RANGE
    assert norm_call(post=0) == ARG                                     # a weight for no norm
    assert norm_call(pre_bias=FAKE) == ARG and norm_call(post_bias=FAKE) == ARG   # biases belong to the layer norm
    assert norm_call(gate_kind=1) == ARG and norm_call(gate=FAKE) == ARG
    assert norm_call(x=None) == ARG and norm_call(h=None) == ARG
    assert norm_call(h_dtype=E4M3) == ARG and norm_call(scale=FAKE) == ARG
    for field in ("x", "residual", "y", "h"):
        assert norm_call(**{field: FAKE + 1}) == ARG
    for field in ("post_weight", "pre_weight"):
        assert norm_call(**{field: FAKE + 2}) == ARG
    assert norm_call(gate_kind=2, gate=FAKE + 2) == ARG
    for field in ("ldx", "ldr", "ldy", "ldh"):
        assert norm_call(**{field: 99}) == SHAPE
    assert norm_call(ldy=120) == SHAPE                                  # in place with another stride
    assert norm_call(t=0, x=None, h=None, y=None, residual=None) == OK


def test_token_logprobs_refuses():
    def call(t=2, v=500, x=f, dt=BF16, ld=500, tg=f, bits=64, it=1.0, top=3, lp=f, en=f, rk=f, ids=f, best=f, ws=f, wsb=1 << 40):
        return L.mbq_token_logprobs(t, v, x, dt, ld, tg, bits, it, top, lp, en, rk, ids, best, ws, wsb, None)

    assert call(t=-1) == SHAPE and call(v=0) == SHAPE and call(v=(1 << 28) + 1) == SHAPE and call(ld=499) == SHAPE
    assert call(top=-1) == SHAPE and call(top=65) == SHAPE and call(v=2, ld=2) == SHAPE
    assert call(dt=E4M3) == ARG and call(dt=8) == ARG and call(bits=16) == ARG
    for it in (0.0, -1.0, 1e31, float("nan"), float("inf")):
        assert call(it=it) == RANGE
    for name in ("x", "tg", "lp", "en", "rk", "ids", "best"):
        assert call(**{name: None}) == ARG
        assert call(**{name: P(FAKE + 1)}) == ARG
    n = ctypes.c_size_t(0)
    assert L.mbq_token_logprobs_workspace(1, 1 << 19, 20, ctypes.byref(n)) == OK and n.value > 0
    for ws, wsb in ((None, 0), (f, n.value - 1), (P(FAKE + 16), n.value)):
        assert call(t=1, v=1 << 19, ld=1 << 19, top=20, ws=ws, wsb=wsb) == WS
    assert L.mbq_token_logprobs_workspace(1, 10, 11, ctypes.byref(n)) == SHAPE
    assert L.mbq_token_logprobs_workspace(1, 10, 1, None) == ARG
    assert call(t=0, x=None, tg=None, lp=None, en=None, rk=None, ids=None, best=None, ws=None, wsb=0) == OK


# --- the Python binding: the library's compute calls replaced by a recorder, CPU tensors in
# --- place of device tensors

class Recorder:
    COMPUTE = {"mbq_fp8_pack", "mbq_fp8_quantize", "mbq_fp8_linear", "mbq_fp8_gated", "mbq_block_norm", "mbq_token_logprobs"}

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        if name not in self.COMPUTE:
            return getattr(self.lib, name)

        def call(*args):
            self.calls.append(name)
            return 0
        return call


class Dev(torch.Tensor):
    """A CPU tensor that says it is on the GPU."""
    is_cuda = True


def D(t):
    return t.as_subclass(Dev)


@pytest.fixture
def rec(monkeypatch):
    r = Recorder(L)
    monkeypatch.setattr(_lib, "LIB", r)
    monkeypatch.setattr(api, "_stream_of", lambda x: None)
    return r


bf, f32, i64 = torch.bfloat16, torch.float32, torch.int64
F8 = torch.float8_e4m3fn


def packed(n=64, k=256, gated=False):
    d = api.fp8_describe(n, k, gated)
    return api.Fp8Linear(d, D(torch.zeros(int(d.total_bytes), dtype=torch.uint8)))


def z(*shape, dt=bf):
    return D(torch.zeros(shape, dtype=dt))


def test_binding_forwards(rec):
    api.fp8_linear(packed(), z(3, 256), y=z(3, 64), workspace=z(1 << 16, dt=torch.uint8))
    api.fp8_gated(packed(gated=True), z(3, 256), y=z(3, 64), workspace=z(1 << 16, dt=torch.uint8))
    api.fp8_linear(packed(), D(torch.zeros(3, 256, dtype=F8)), z(2, 3, dt=f32), y=z(3, 64))
    api.fp8_quantize(z(3, 300), q=D(torch.zeros(3, 300, dtype=F8)), scale=z(3, 3, dt=f32))
    api.block_norm(z(3, 300), z(3, 300), pre=z(300, dt=f32), y=z(3, 300), h=z(3, 300))
    assert rec.calls == ["mbq_fp8_linear", "mbq_fp8_gated", "mbq_fp8_linear", "mbq_fp8_quantize", "mbq_block_norm"]


REFUSED = [
    lambda: api.fp8_linear(packed(), torch.zeros(3, 256, dtype=bf)),                       # a CPU tensor
    lambda: api.fp8_linear(packed(), z(3, 255)),                                           # wrong inputs
    lambda: api.fp8_linear(packed(), z(3, 256, dt=torch.float16)),
    lambda: api.fp8_linear(packed(), z(256)),
    lambda: api.fp8_linear(packed(), z(256, 3).t()),                                       # columns apart
    lambda: api.fp8_linear(packed(), D(torch.zeros(1, 256, dtype=bf).expand(3, 256))),     # rows on top of each other
    lambda: api.fp8_linear(packed(gated=True), z(3, 256)),
    lambda: api.fp8_gated(packed(), z(3, 256)),
    lambda: api.fp8_gated(packed(gated=True), z(3, 256), act="relu"),
    lambda: api.fp8_linear(packed(), z(3, 256), z(2, 3, dt=f32)),                          # a scale without codes
    lambda: api.fp8_linear(packed(), D(torch.zeros(3, 256, dtype=F8)), z(3, 2, dt=f32)),   # the scale transposed
    lambda: api.fp8_linear(packed(), z(3, 256), y=z(3, 63), workspace=z(1 << 16, dt=torch.uint8)),
    lambda: api.fp8_linear(packed(), z(3, 256), y=z(3, 64, dt=torch.float16)),
    lambda: api.fp8_linear(packed(), z(32, 256), y=z(32, 64), workspace=z(8, dt=torch.uint8)),
    lambda: api.fp8_linear(api.Fp8Linear(packed().desc, z(100, dt=torch.uint8)), z(3, 256)),
    lambda: api.fp8_quantize(z(3, 300), q=D(torch.zeros(3, 299, dtype=F8))),
    lambda: api.fp8_quantize(z(3, 300), q=D(torch.zeros(3, 300, dtype=F8)), scale=z(3, 2, dt=f32)),
    lambda: api.fp8_pack(z(64, 256), z(1, 2, dt=f32)),                                     # scales for what is quantized here
    lambda: api.fp8_pack(D(torch.zeros(64, 256, dtype=F8))),                               # codes without scales
    lambda: api.fp8_pack(D(torch.zeros(64, 256, dtype=F8)), z(1, 3, dt=f32)),
    lambda: api.fp8_pack(z(64, 256, dt=torch.float16)),
    lambda: api.fp8_pack_gated(z(64, 256), z(64, 128)),
    lambda: api.fp8_pack(z(64, 256), out=z(100, dt=torch.uint8)),
    lambda: api.block_norm(z(3, 300), z(3, 299)),
    lambda: api.block_norm(z(3, 300), kind="batch"),
    lambda: api.block_norm(z(3, 300), pre=z(300)),                                         # weights are float32
    lambda: api.block_norm(z(3, 300), pre=z(299, dt=f32)),
    lambda: api.block_norm(z(3, 300), gate=z(4, dt=f32)),
    lambda: api.block_norm(z(3, 300), gate=z(3, 300, dt=f32)),                             # a full gate has x's type
    lambda: api.block_norm(z(3, 300), z(3, 300), y=z(3, 300, dt=f32), h=z(3, 300)),        # y has residual's type
    lambda: api.block_norm(z(3, 300), y=z(3, 300), h=z(3, 300), scale=z(3, 3, dt=f32)),
    lambda: api.block_norm(z(3, 300), y=z(3, 300), h=z(3, 300), quantized=True),
    lambda: api.token_logprobs(z(3, 300), z(4, dt=i64)),
    lambda: api.token_logprobs(z(3, 300), z(3, dt=f32)),
    lambda: api.token_logprobs(z(3, 300), z(3, dt=i64), top=65),
    lambda: api.token_logprobs(z(3, 30), z(3, dt=i64), top=31),
    lambda: api.token_logprobs(z(3, 30), z(3, dt=i64), top=-1),
    lambda: api.token_logprobs(z(300, 3).t(), z(3, dt=i64)),
]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_binding_refuses(rec, i):
    with pytest.raises((TypeError, ValueError)):
        REFUSED[i]()
    assert rec.calls == []
