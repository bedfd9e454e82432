"""The fp64 statements of the MLP-block operators against differences, hand
values and their definitions (CPU)."""
import math

import numpy as np
import pytest

from oracle import mlp


def _diff(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(0)
    s, w, dy = rng.normal(size=(3, 17)), rng.normal(size=17), rng.normal(size=(3, 17))
    eps = 1e-3
    ds, dw = mlp.norm_backward(dy, s, w, mlp.rstd(s, eps), np.zeros_like(s))
    for _ in range(4):
        d, e = rng.normal(size=s.shape), rng.normal(size=w.shape)
        # central differences: truncation h^2 |f'''| / 6 ~ 1e-9, rounding 1e-15 / h ~ 1e-10
        assert abs(np.sum(ds * d) - _diff(lambda v: np.sum(dy * mlp.norm(v, w, eps)), s, d)) < 1e-7
        assert abs(np.sum(dw * e) - _diff(lambda v: np.sum(dy * mlp.norm(s, v, eps)), w, e)) < 1e-7


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gated_gradients_against_differences(kind):
    rng = np.random.default_rng(1)
    x, wg, wu = rng.normal(size=(2, 5)), rng.normal(size=(7, 5)), rng.normal(size=(7, 5))
    bg, bu, dh = rng.normal(size=7), rng.normal(size=7), rng.normal(size=(2, 7))
    g, u, _ = mlp.gated(x, wg, wu, bg, bu, kind)
    dx, dg, du = mlp.gated_backward(dh, g, u, wg, wu, kind)
    for _ in range(4):
        d, e = rng.normal(size=x.shape), rng.normal(size=7)
        assert abs(np.sum(dx * d) - _diff(
            lambda v: np.sum(dh * mlp.gated(v, wg, wu, bg, bu, kind)[2]), x, d)) < 1e-7
        assert abs(np.sum(dg * e) - _diff(
            lambda v: np.sum(dh * mlp.gated(x, wg, wu, v, bu, kind)[2]), bg, e)) < 1e-7
        assert abs(np.sum(du * e) - _diff(
            lambda v: np.sum(dh * mlp.gated(x, wg, wu, bg, v, kind)[2]), bu, e)) < 1e-7


def test_act_hand_values():
    f, d = mlp.act(np.array([0.0, 1.0, -800.0, 800.0]), "silu")
    assert np.allclose(f, [0.0, 1 / (1 + math.exp(-1)), 0.0, 800.0], atol=1e-12)
    assert np.allclose(d[[0, 2, 3]], [0.5, 0.0, 1.0], atol=1e-12)
    f, d = mlp.act(np.array([0.0, -800.0, 800.0]), "gelu_tanh")
    assert np.allclose(f, [0.0, 0.0, 800.0]) and np.allclose(d, [0.5, 0.0, 1.0])


def test_checkpoint_hand_values():
    # scale 254 / 127 = 2: 5 / 2 = 2.5 and 3 / 2 = 1.5 are ties, to even
    x = np.zeros((2, 70))
    x[0, :5] = [254.0, 5.0, -5.0, 3.0, 1.0]
    x[0, 64] = -127.0
    q, s = mlp.checkpoint(x)
    assert q[0, :5].tolist() == [127, 2, -2, 2, 0] and q[0, 64] == -127
    assert s[0].tolist() == [2.0, 1.0] and s[1].tolist() == [0.0, 0.0] and not q[1].any()
    assert np.array_equal(mlp.restore(q, s)[0, :5], [254.0, 4.0, -4.0, 4.0, 0.0])


def test_checkpoint_is_half_a_step_off():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(5, 333))
    q, s = mlp.checkpoint(x)
    step = np.repeat(s.astype(np.float64), 64, axis=1)[:, :333]
    assert np.all(np.abs(mlp.restore(q, s) - x) <= 0.5 * step * (1 + 1e-6))


def test_row_codes():
    v = np.array([[1.0, -127.0, 0.5, 1.5], [0.0, 0.0, 0.0, 0.0]])
    q, s = mlp.row_codes(v)
    assert q.tolist() == [[1, -127, 0, 2], [0, 0, 0, 0]] and s.tolist() == [1.0, 0.0]
