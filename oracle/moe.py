"""Plain NumPy statement, in fp64, of a mixture-of-experts layer: the router's
choice, the chosen experts' gated pairs and down projections, and their sum."""
import numpy as np

from .mlp import act


def route(x, router, topk, score="softmax", norm=True):
    """(ids [M, topk], weights [M, topk]): the experts of the largest logits,
    falling, the lower index among equals; a NaN logit is never taken (ids of -1
    and weights of 0 where numbers run out), an infinite one is a number like others
    (a softmax whose largest logit is infinite is NaN)."""
    with np.errstate(invalid="ignore"):
        return _route(x @ router.T, topk, score, norm)


def _route(logits, topk, score, norm):
    M, E = logits.shape
    ids, w = np.full((M, topk), -1), np.zeros((M, topk))
    for m in range(M):
        ok = [e for e in range(E) if logits[m, e] == logits[m, e]]
        order = sorted(ok, key=lambda e: (-logits[m, e], e))[:topk]
        if not order:
            continue
        top = logits[m, order[0]]
        total = sum(np.exp(logits[m, e] - top) for e in ok)
        for i, e in enumerate(order):
            ids[m, i] = e
            w[m, i] = np.exp(logits[m, e] - top) / total if score == "softmax" else 1 / (1 + np.exp(-logits[m, e]))
    if norm:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=(ids >= 0) & (total != 0))
    return ids, w


def layer(x, ids, weights, gate, up, down, kind):
    """y [M, K] from stacked gate and up [E, inner, K] and down [E, K, inner]."""
    y = np.zeros((x.shape[0], x.shape[1]))
    for m in range(x.shape[0]):
        for e, w in zip(ids[m], weights[m]):
            if 0 <= e < gate.shape[0]:
                h = act(gate[e] @ x[m], kind)[0] * (up[e] @ x[m])
                y[m] += w * (down[e] @ h)
    return y
