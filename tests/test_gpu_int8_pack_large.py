"""Packing as many outputs as mbq_int8_describe accepts: 17 weights of 2^24 outputs are 17 * 2^20 groups of 16 rows, and a
workgroup of 256 threads for each would be 2^32 threads and more.  A launch takes their number modulo 2^32 without an error, so
that only the first weight would be packed."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import expert_oracle as E
from test_gpu_int8_linear import DEV, api   # noqa: F401

pytestmark = pytest.mark.gpu
EXPERTS, N = 17, 1 << 24


def test_launch_limit_is_passed():
    assert EXPERTS * (N // 16) * 256 >= 1 << 32


@pytest.mark.parametrize("source", ["codes", "bf16"])
def test_pack(api, source):
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB")
    at = torch.arange(EXPERTS * N, dtype=torch.int32, device=DEV)
    if source == "codes":
        w, scale = (at % 255 - 127).to(torch.int8), at.float()
        p = api.expert_pack(w.view(EXPERTS, N, 1), scale.view(EXPERTS, N))
        want = w
    else:                                                    # a row of one element: its code is 127 or -127, its scale |w| / 127
        w = (at % 251 - 125).to(torch.bfloat16)
        p = api.expert_pack(w.view(EXPERTS, N, 1))
        codes, scales = E.quantize(np.arange(-125, 126, dtype=np.float32)[:, None])
        want, scale = (torch.from_numpy(v).to(DEV)[at % 251] for v in (codes[:, 0], scales))
    del at
    d = p.desc
    assert d.row_blocks == N // 16 and d.k_blocks == 1
    tiles = p.blob[: d.scales_offset].view(torch.int8).view(-1, 2048)
    assert torch.equal(tiles[:, : 16 * 16 : 16], want.view(-1, 16))            # code of row r at byte 16 r of the tile
    for lo in range(0, tiles.shape[0], 1 << 21):                               # and every other byte 0
        band = tiles[lo : lo + (1 << 21)]
        assert int(band.count_nonzero()) == int(want.view(-1, 16)[lo : lo + (1 << 21)].count_nonzero())
    got = p.blob[d.scales_offset : d.scales_offset + 4 * EXPERTS * N].view(torch.float32)
    assert torch.equal(got, scale)
