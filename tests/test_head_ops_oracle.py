"""The oracle of the operators around the head, pinned on its own: closed forms, differences."""
import numpy as np
import pytest

from oracle import head_ops_oracle as HO


def test_entropy_and_alternatives_of_closed_forms():
    # equal logits: entropy log V, alternatives in rising id, each log-prob -log V
    o = HO.token_stats(np.zeros((2, 3)), np.ones((7, 3)), [0, 6], n_top=9)
    assert np.allclose(o["entropy"], np.log(7)) and np.allclose(o["logp"], -np.log(7))
    assert o["top_ids"][0].tolist() == [0, 1, 2, 3, 4, 5, 6, -1, -1]
    assert np.all(np.isneginf(o["top_logp"][:, 7:]))
    # two logits a, 0: p = sigmoid(a), entropy the binary one
    a = 1.7
    o = HO.token_stats(np.array([[1.0]]), np.array([[a], [0.0]]), [1], n_top=2)
    p = 1 / (1 + np.exp(-a))
    assert np.isclose(o["entropy"][0], -p * np.log(p) - (1 - p) * np.log(1 - p))
    assert o["top_ids"].tolist() == [[0, 1]] and np.isclose(o["logp"][0], np.log(1 - p))
    # a bad target scores 0
    assert HO.token_stats(np.ones((1, 1)), np.ones((2, 1)), [2])["logp"][0] == 0


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradients_are_the_forwards_differences(kind):
    rng = np.random.default_rng(1)
    x, w, b = rng.normal(size=(3, 8)), rng.normal(size=8), rng.normal(size=8)
    dy = rng.normal(size=(3, 8))

    def f(x, w, b):
        return float((HO.norm_forward(x, w, b, kind)[0] * dy).sum())

    _, mean, rstd = HO.norm_forward(x, w, b, kind)
    got = HO.norm_backward(x, dy, mean, rstd, w, kind)
    h = 1e-6
    for k, g in enumerate(got):
        args = [x, w, b]
        for i in np.ndindex(args[k].shape):
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[k][i] += h
            down[k][i] -= h
            # central difference: error about h^2 plus 1e-16 / h, both below 1e-8
            assert abs((f(*up) - f(*down)) / (2 * h) - g[i]) < 1e-7


def test_layer_norm_statistics():
    x = np.random.default_rng(2).normal(3.0, 2.0, (4, 64))
    y, mean, rstd = HO.norm_forward(x, eps=0.0)
    assert np.allclose(y.mean(axis=1), 0) and np.allclose((y * y).mean(axis=1), 1)
    y, _, _ = HO.norm_forward(x, kind="rms", eps=0.0)
    assert np.allclose((y * y).mean(axis=1), 1)


def test_checkpoint_scale_and_rounding():
    x = np.zeros((1, 96))
    x[0, 0] = 127.0            # exactly 127 * 2^0
    x[0, 32] = 127.5           # one step above: the exponent moves up
    x[0, 33] = 3.0             # 1.5 steps of 2: half to even
    x[0, 64] = np.inf
    codes, scales, values = HO.checkpoint(x)
    assert scales.tolist() == [[127, 128, 255]]
    assert codes[0, 0] == 127 and codes[0, 32] == 64 and codes[0, 33] == 2
    assert values[0, 32] == 128.0 and np.isnan(values[0, 64:]).all()


def test_checkpoint_error_bound_and_bf16_exactness():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(5, 72)) * 2.0 ** rng.integers(-30, 30, (5, 72))
    codes, scales, values = HO.checkpoint(x)
    step = 2.0 ** (np.repeat(scales.astype(np.float64), 32, axis=1)[:, :72] - 127)
    assert np.all(np.abs(values - x) <= step / 2)
    bits = values.astype(np.float32).view(np.uint32)
    assert np.all(bits & 0xFFFF == 0) and np.all(values.astype(np.float32) == values)
    # nothing smaller holds the block
    top = np.abs(x[:, :64].reshape(5, 2, 32)).max(axis=2)
    assert np.all(top > 127 * 2.0 ** (scales[:, :2].astype(np.float64) - 128))
