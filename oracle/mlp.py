"""Plain NumPy statements, in fp64, of the operators around the packed layers:
RMS norm with the residual's addition, 8-bit activation checkpoints, the
gated pair of projections, and their gradients.

Inputs are fp64 arrays of the values that the device holds (decoded from
their 16 bits); weights are the dequantized matrices of dequant_f64.
"""
import numpy as np

GROUP = 64


def rstd(s, eps):
    return 1.0 / np.sqrt(np.mean(s * s, axis=-1, keepdims=True) + eps)


def norm(s, weight, eps):
    """s * weight * rstd, before any rounding."""
    return s * weight * rstd(s, eps)


def norm_backward(dy, s, weight, r, ds_in):
    """(ds, dweight) with r [M, 1] the forward's rstd."""
    xh = s * r
    g = dy * weight
    c = np.mean(g * xh, axis=-1, keepdims=True)
    return r * (g - xh * c) + ds_in, np.sum(dy * xh, axis=0)


def row_codes(v):
    """int8 row and its scale: ys = fl32(max|v| / 127), rint(v / ys)."""
    ys = (np.max(np.abs(v), axis=-1, keepdims=True) / 127.0).astype(np.float32)
    return _codes(v, ys), ys[..., 0]


def _codes(v, sc):
    d = sc.astype(np.float64)
    q = np.divide(v, d, out=np.zeros_like(v), where=d > 0)
    return np.clip(np.rint(q), -127, 127).astype(np.int8)


def checkpoint(x):
    """(codes int8 [M, K], scales fp32 [M, ceil(K / 64)])."""
    M, K = x.shape
    n = -(-K // GROUP)
    p = np.zeros((M, n * GROUP))
    p[:, :K] = x
    g = p.reshape(M, n, GROUP)
    sc = (np.max(np.abs(g), axis=-1) / 127.0).astype(np.float32)
    return _codes(g, sc[..., None]).reshape(M, -1)[:, :K].copy(), sc


def restore(codes, scales):
    K = codes.shape[1]
    return codes.astype(np.float64) * np.repeat(scales.astype(np.float64), GROUP, axis=1)[:, :K]


def act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        s = 0.5 * (1.0 + np.tanh(0.5 * g))
        return g * s, s + g * s * (1.0 - s)
    a, b = np.sqrt(2.0 / np.pi), 0.044715
    t = np.tanh(a * (g + b * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * a * (1 + 3 * b * g * g)


def gated(x, wg, wu, bg, bu, kind):
    """(g, u, h) of h = act(x Wg^T + bg) * (x Wu^T + bu)."""
    g, u = x @ wg.T + bg, x @ wu.T + bu
    return g, u, act(g, kind)[0] * u


def gated_backward(dh, g, u, wg, wu, kind):
    """(dx, dg, du)."""
    f, d = act(g, kind)
    dg, du = dh * u * d, dh * f
    return dg @ wg + du @ wu, dg, du
