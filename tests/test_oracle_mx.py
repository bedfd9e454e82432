"""Pins of the MXFP4 and mixture-of-experts statements (CPU)."""
import numpy as np
import pytest

from oracle import moe, mx


def test_values_and_scales_by_hand():
    x = np.zeros((1, 64))
    x[0, :9] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0]     # scale 1: every border
    x[0, 32:36] = [7.9, -1.0, 0.4, -0.0]                               # scale 1 again: 7.9 stops at 6
    c, s = mx.quantize(x)
    assert s.tolist() == [[127, 127]]
    assert c[0, :9].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 14]
    assert c[0, 32:36].tolist() == [7, 10, 1, 8]
    v = mx.dequantize(c, s)
    assert v[0, :9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -4] and v[0, 32:35].tolist() == [6, -1, 0.5]


@pytest.mark.parametrize("top,byte", [(1.0, 125), (1.99, 125), (2.0, 126), (4.0, 127), (2.0 ** 127, 252),
                                      (2.0 ** -124, 1), (2.0 ** -125, 0), (2.0 ** -149, 0), (0.0, 0)])
def test_scale_bytes(top, byte):
    x = np.zeros((1, 32))
    x[0, 5] = -top
    assert mx.quantize(x)[1][0, 0] == byte


def test_not_finite_and_words():
    x = np.ones((3, 32))
    x[0, 3], x[1, 31] = np.nan, -np.inf
    c, s = mx.quantize(x)
    assert s[:, 0].tolist() == [255, 255, 125] and not c[:2].any()
    d = mx.dequantize(c, s)
    assert np.isnan(d[:2]).all() and (d[2] == 1).all()
    assert mx.pack(np.arange(16, dtype=np.uint8)[None])[0].tolist() == [0x76543210, 0xFEDCBA98]


def test_every_code_comes_back_and_is_nearest():
    rng = np.random.default_rng(0)
    for s in (0, 1, 100, 127, 252):
        c = np.tile(np.arange(16, dtype=np.uint8), 2)[None]
        back, sb = mx.quantize(mx.dequantize(c, np.array([[s]], np.uint8)))
        assert np.array_equal(back, c) and sb[0, 0] == s
    x = rng.normal(size=(50, 64)) * 10.0 ** rng.uniform(-30, 30, size=(50, 1))
    c, s = mx.quantize(x)
    unit = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    err = np.abs(mx.dequantize(c, s) - x) / unit
    # half the grid's step where a value lies, and what the largest lose at 6
    a = np.abs(x) / unit
    assert np.all(err <= np.where(a > 6, a - 6, np.where(a >= 4, 1.0, np.where(a >= 2, 0.5, 0.25))) + 1e-12)
    assert a.max() < 8


def test_route_by_hand():
    x, r = np.eye(3), np.array([[0.0, 1.0, np.nan], [2.0, 1.0, 1.0], [2.0, 3.0, np.nan], [-1.0, 1.0, 0.0]])
    ids, w = moe.route(x, np.nan_to_num(r), 2)
    assert ids.tolist() == [[1, 2], [2, 0], [1, 0]]
    assert np.allclose(w[0], 0.5) and np.allclose(w.sum(1), 1)
    ids, w = moe.route(x, np.nan_to_num(r), 2, score="sigmoid", norm=False)
    assert np.allclose(w[1], [1 / (1 + np.exp(-3.0)), 1 / (1 + np.exp(-1.0))])
    # NaN logits run out of numbers
    ids, w = moe.route(np.array([[1.0]]), np.array([[np.nan], [1.0], [np.nan]]), 2)
    assert ids.tolist() == [[1, -1]] and w.tolist() == [[1.0, 0.0]]


def test_layer_is_the_weighted_sum():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(2, 4))
    g, u, d = rng.normal(size=(3, 6, 4)), rng.normal(size=(3, 6, 4)), rng.normal(size=(3, 4, 6))
    y = moe.layer(x, np.array([[2, -1], [0, 0]]), np.array([[0.5, 9.0], [0.25, 0.5]]), g, u, d, "silu")
    h = (g[2] @ x[0]) / (1 + np.exp(-(g[2] @ x[0]))) * (u[2] @ x[0])
    assert np.allclose(y[0], 0.5 * (d[2] @ h))
    h = (g[0] @ x[1]) / (1 + np.exp(-(g[0] @ x[1]))) * (u[0] @ x[1])
    assert np.allclose(y[1], 0.75 * (d[0] @ h))


def test_route_with_infinite_logits():
    x, r = np.array([[1.0]]), np.array([[2.0], [-np.inf], [1.0], [np.nan]])
    for norm in (False, True):
        ids, w = moe.route(x, r, 4, norm=norm)
        assert ids.tolist() == [[0, 2, 1, -1]] and np.allclose(w[0, :2], [1 / (1 + np.exp(-1)), 1 / (1 + np.e)])
        assert w[0, 2:].tolist() == [0, 0]
    ids, w = moe.route(x, np.array([[np.inf], [1.0], [np.nan]]), 3)
    assert ids.tolist() == [[0, 1, -1]] and np.isnan(w[0, :2]).all() and w[0, 2] == 0
    ids, w = moe.route(x, np.array([[-np.inf], [-np.inf]]), 2, score="sigmoid")
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0, 0]]
