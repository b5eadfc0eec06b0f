"""Codes of rows that hold a NaN with any payload, of either sign, or an infinity: all 0, with the scale NaN; other rows as
the oracle has them.  Codes and scales are exact, so nothing has a tolerance."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import expert_oracle as E
from test_gpu_int8_linear import DEV, DT, api   # noqa: F401

pytestmark = pytest.mark.gpu
# float32 bits: quiet and signalling NaN of both signs with every kind of low byte, the plain NaN, the infinities
BAD = (0x7FC00001, 0xFFC000FF, 0x7F800001, 0xFF8000AA, 0x7FFFFFFF, 0xFFFFFF80, 0x7FC00000, 0xFFC00000, 0x7F800000, 0xFF800000)


def rows_with_bad(k, dtype, seed):
    """(x [2 len(BAD) + 1, k], which rows are good): a bad element at a random place of every other row."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((2 * len(BAD) + 1, k)).astype(np.float32)
    bits = x.view(np.uint32)
    for i, b in enumerate(BAD):
        bits[2 * i + 1, rng.integers(0, k)] = b
    x = torch.from_numpy(bits.view(np.int32)).to(DEV).view(torch.float32)
    if dtype == "bf16":                                      # the upper half of the bits, so that payloads stay
        x = (x.view(torch.int32) >> 16).to(torch.int16).view(torch.bfloat16)
        # the low halves that made a NaN are gone: such a row holds an infinity
    return x, torch.isfinite(x.float()).all(1).cpu().numpy()


# one, four and sixteen waves a row, rows held in registers and rows read again, a part of a piece at the end
@pytest.mark.parametrize("k", [1, 7, 300, 2048, 2051, 8200, 40001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize(api, k, dtype):
    x, good = rows_with_bad(k, dtype, k)
    assert good.sum() == len(BAD) + 1
    q, s = (v.cpu().numpy() for v in api.int8_quantize(x))
    assert (q[~good] == 0).all() and np.isnan(s[~good]).all()
    codes, scale = E.quantize(x[torch.from_numpy(good).to(DEV)].float().cpu().numpy())
    assert np.array_equal(q[good], codes) and np.array_equal(s[good], scale)


@pytest.mark.parametrize("k", [7, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pack(api, k, dtype):
    w, good = rows_with_bad(k, dtype, k + 1)
    n = w.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = api.int8_pack(w, status=status)
    d = p.desc
    blob = p.blob.cpu().numpy()
    tiles = blob[: d.scales_offset].view(np.int8).reshape(d.row_blocks, d.k_blocks, 2, 4, 16, 16)   # rb, kb, half, c, r, byte
    codes = tiles.transpose(0, 4, 1, 2, 3, 5).reshape(d.row_blocks * 16, d.k_blocks * 128)
    scale = blob[d.scales_offset :].view(np.float32)[:n]
    assert int(status) == 1
    assert (codes[:n][~good] == 0).all() and np.isnan(scale[~good]).all()
    want, want_s = E.quantize(w[torch.from_numpy(good).to(DEV)].float().cpu().numpy())
    assert np.array_equal(codes[:n][good, :k], want) and np.array_equal(scale[good], want_s)
    assert (codes[n:] == 0).all() and (codes[:, k:] == 0).all()


@pytest.mark.parametrize("t", [1, 5, 21])
def test_linear(api, t):
    """Outputs of such rows are NaN, of the others untouched, on every path of the quantization."""
    x, good = rows_with_bad(300, "f32", 3)
    x, good = x[:t], good[:t]
    w = torch.randn(50, 300, device=DEV)
    p = api.int8_pack(w)
    y = api.int8_linear(p, x).cpu().numpy()
    assert np.isnan(y[~good]).all()
    xq, xs = E.quantize(x.cpu().numpy()[good])
    wq, ws = E.quantize(w.cpu().numpy())
    ref, _ = E.product(xq, xs, wq, ws)
    assert (np.abs(y[good] - ref) <= np.abs(ref) * 2.0 ** -22 + 1e-38).all()   # three roundings of 2^-24
