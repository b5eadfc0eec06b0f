"""Arguments of the dense operators that the Python wrapper has to name itself (no GPU): the
library's compute calls replaced by a recorder, CPU tensors in place of device tensors."""
import pytest

torch = pytest.importorskip("torch")

from test_dense_validation import D, api, bf, f32, packed, rec, z   # noqa: E402,F401


@pytest.mark.parametrize("gated", [False, True])
def test_a_blob_lies_in_one_piece(rec, gated):
    p = packed(gated=gated)
    apart = api.Fp8Linear(p.desc, D(torch.zeros(2 * p.blob.numel(), dtype=torch.uint8)[::2]))
    with pytest.raises(ValueError, match="contiguous"):
        (api.fp8_gated if gated else api.fp8_linear)(apart, z(3, 256), y=z(3, 64))
    assert rec.calls == []


@pytest.mark.parametrize("gate", [0.5, [1.0, 2.0, 3.0]])
def test_a_gate_is_a_tensor(rec, gate):
    with pytest.raises(TypeError, match="gate must be a tensor"):
        api.block_norm(z(3, 300), gate=gate, y=z(3, 300), h=z(3, 300))
    assert rec.calls == []
