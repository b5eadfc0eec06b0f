"""The dense operators' oracle pinned to hand-worked values and to independent statements of
the same formulas (no GPU)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import dense_oracle as D


def test_e4m3_table():
    v = D.e4m3_values()
    assert v[0x38] == 1.0 and v[0x7E] == 448.0 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0xB8] == -1.0
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(v, t.astype(np.float64), equal_nan=True)


def test_e4m3_rounding():
    v = np.array([1.0625, 1.1875, 1.06251, 464 - 1e-9, 2.0 ** -10, 1.5 * 2.0 ** -9, -0.0, 0.0, np.nan])
    assert D.e4m3_encode(v).tolist() == [0x38, 0x3A, 0x39, 0x7E, 0x00, 0x02, 0x80, 0x00, 0x7F]
    x = np.random.default_rng(0).standard_normal(4000).astype(np.float32) * 100
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(D.e4m3_encode(x), t)


def test_quantize_by_hand():
    x = np.zeros((2, 130), np.float32)
    x[0, :3] = [4.48, -2.24, 0.0112]
    x[0, 129] = -896.0
    codes, scale = D.quantize(x)
    assert scale.shape == (2, 2) and abs(scale[0, 0] - 0.01) < 1e-9 and scale[1, 0] == 2.0
    assert scale[0, 1] == np.float32(2.0 ** -96) / np.float32(448) and not codes[1].any()
    assert codes[0, :3].tolist() == [0x7E, 0xF6, 0x39 if codes[0, 2] == 0x39 else 0x3A] and codes[0, 129] == 0xFE
    v = D.values_x(codes, scale)
    assert np.abs(v - x).max() <= 896 / 16


def test_weight_blocks():
    w = np.zeros((130, 200), np.float32)
    w[0, 0], w[129, 199], w[129, 0] = 448.0, 3.5, -3.5
    codes, scale = D.quantize_weight(w)
    assert scale.shape == (2, 2) and scale[0, 0] == 1.0 and scale[1, 0] == np.float32(3.5) / np.float32(448)
    assert np.array_equal(D.values_w(codes, scale)[[0, 129]][:, [0, 199]], [[448.0, 0], [-3.5, 3.5]])


def test_norms():
    x = np.array([[3.0, -1.0, 2.0, 0.0]])
    n, _ = D.norm(x, None, None, "rms", 0.0)
    assert np.allclose(n, x / np.sqrt(3.5))
    n, _ = D.norm(x, np.full(4, 2.0), np.ones(4), "layer", 0.0)
    assert np.allclose(n, (x - 1) / np.sqrt(2.5) * 2 + 1)
    y, h, _, _ = D.block_norm(x, 2 * x, None, None, 0.5, 3.0, 4.0, 0.0, "rms")
    assert np.allclose(y, 8 * x) and np.allclose(h, x / np.sqrt(3.5))
    t = torch.randn(5, 33, dtype=torch.float64)
    w, b = torch.randn(33, dtype=torch.float64), torch.randn(33, dtype=torch.float64)
    assert np.allclose(D.norm(t.numpy(), w.numpy(), b.numpy(), "layer", 1e-5)[0],
                       torch.nn.functional.layer_norm(t, (33,), w, b, 1e-5).numpy())


def test_activations():
    g = torch.linspace(-9, 9, 101, dtype=torch.float64)
    assert np.allclose(D.act(g.numpy(), "silu"), torch.nn.functional.silu(g).numpy())
    assert np.allclose(D.act(g.numpy(), "gelu_tanh"), torch.nn.functional.gelu(g, approximate="tanh").numpy())


def test_logprobs():
    z = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.2, 0.7]]))
    lp, ent, rank, ids, best = D.token_logprobs(z, [2, 9], 2, 1.0)
    assert np.allclose(lp, [np.log(0.25), 0]) and rank.tolist() == [3, 0] and ids.tolist() == [[0, 1], [2, 1]]
    assert np.allclose(ent, [1.5 * np.log(2), -(0.1 * np.log(0.1) + 0.2 * np.log(0.2) + 0.7 * np.log(0.7))])
    assert np.allclose(np.exp(best), [[0.5, 0.25], [0.7, 0.2]])
    t = torch.randn(6, 50, dtype=torch.float64)
    d = torch.distributions.Categorical(logits=t * 0.7)
    lp, ent, rank, ids, best = D.token_logprobs(t.numpy(), [3] * 6, 0, 0.7)
    assert np.allclose(lp, d.log_prob(torch.tensor([3] * 6)).numpy()) and np.allclose(ent, d.entropy().numpy())
    lp, ent, rank, ids, best = D.token_logprobs(np.array([[-np.inf] * 3, [np.nan, 0, 0]]), [1, 1], 1, 1.0)
    assert lp[0] == -np.inf and ent[0] == 0 and rank.tolist() == [2, 0] and ids.tolist() == [[0], [-1]] and np.isnan(lp[1])
