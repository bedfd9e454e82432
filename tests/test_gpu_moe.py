"""GPU parity of mixture-of-experts layers with their fp64 statement.

Tolerances.  The router's logits are held in fp64: the
choice is the statement's.  An expert's product: 36 roundings of 2^-24 (32
additions, the chunk's two fused steps, their sum) of a chunk's magnitude
sum (MAG + u) |x| S + |T| |x|, whose codes carry MAG = 128 (bf16), 1024 (fp16)
or 0 (MXFP4), then the row's chunks and at most 24 partial sums of at most
sum |x| |w|; taken double for matrix instructions that truncate.
"""
import numpy as np
import pytest

import oracle
from helpers import qformat_of
from oracle import mlp, moe, mx
from test_gpu_mlp import DT, TINY, U, dev, f64, within
from test_gpu_mx import on_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_weight_only_qlinear_amd import qlinear
    return qlinear


def desc(q, fmt, N, K):
    D = q.QDesc
    if fmt.startswith("affine"):
        gs, meta = fmt[6:].split(".")
        return D.affine(N, K, 4, int(gs), meta)
    return {"mxfp4": D.mxfp4, "q4k": D.q4k, "sym4": D.sym4, "sym4.32": lambda n, k: D.sym4(n, k, 32)}[fmt](N, K)


def stack(q, fmt, rng, E, rows, K, dt):
    """A stacked layer: descriptor, buffers, weights [E, rows, K] in fp64 and
    the magnitudes that the chunks' sums pass through."""
    d = desc(q, fmt, E * rows, K)
    W = (rng.normal(size=(E * rows, K)) * 0.08).astype(np.float32)
    if fmt == "mxfp4":
        c, s = mx.quantize(W.astype(np.float64))
        w64 = mx.dequantize(c, s)
        return d, on_gpu(c, s), w64.reshape(E, rows, K), np.abs(w64).reshape(E, rows, K)
    buf = q.qpack_quantize(d, torch.from_numpy(W).cuda())
    f = qformat_of(d)
    w64 = oracle.dequant_f64(oracle.quantize(W, f), f)
    # a scale of its group: what one code step is worth, at most (group range) / 14
    g = d.group_size
    G = w64.reshape(E * rows, K // g, g)
    step = (G.max(-1) - G.min(-1)).clip(min=0) / 7 + np.abs(G).max(-1) / 7
    mag = (2 * (128 if dt == "bf16" else 1024) + 32) * step
    return d, buf, w64.reshape(E, rows, K), np.repeat(mag, g, axis=1).reshape(E, rows, K)


def prod_tol(x, w, mag):
    """Per element of x [n, K] @ w[K].T."""
    K = w.shape[-1]
    return 72 * 2.0 ** -24 * (np.abs(x) @ mag.T) + 2 * (K // 32 + 24) * 2.0 ** -24 * (np.abs(x) @ np.abs(w).T)


def check(o, x64, ids, wts, G, Um, Dn, kind, dt, yd):
    """y within what every rounding on the way can add up to."""
    (gw, gm), (uw, um), (dw, dm) = G, Um, Dn
    M, K = x64.shape
    ref, tol = np.zeros((M, K)), np.zeros((M, K))
    for m in range(M):
        for e, w in zip(ids[m], wts[m]):
            if not 0 <= e < gw.shape[0]:
                continue
            x = x64[m][None]
            g, u = x @ gw[e].T, x @ uw[e].T
            dg, du = prod_tol(x, gw[e], gm[e]), prod_tol(x, uw[e], um[e])
            a = mlp.act(g, kind)[0]
            h = a * u
            # |act'| <= 1.13; the logistic's argument and exponential: 2^-17
            dh = 1.13 * dg * (np.abs(u) + du) + np.abs(a) * du + (U[dt] + 2.0 ** -17) * np.abs(h) + TINY[dt]
            ref[m] += w * (h @ dw[e].T)[0]
            tol[m] += abs(w) * (dh @ np.abs(dw[e]).T + prod_tol(np.abs(h) + dh, dw[e], dm[e]) +
                                2.0 ** -22 * (np.abs(h) @ np.abs(dw[e]).T))[0]
    within(o.y, ref, tol * (1 + U[yd]) + (U[yd] + 2.0 ** -20) * np.abs(ref) + TINY[yd], "y")
    return ref


def parts(s):
    return s[2], s[3]


CASES = [  # M, E, topk, K, inner, up format, down format, dt, y, act, score, norm
    (1, 2, 1, 32, 32, "mxfp4", "mxfp4", "bf16", "f32", "silu", "softmax", True),
    (1, 8, 2, 512, 256, "mxfp4", "mxfp4", "bf16", "bf16", "silu", "softmax", True),
    (3, 5, 3, 544, 96, "mxfp4", "mxfp4", "f16", "f16", "gelu_tanh", "sigmoid", True),
    (7, 4, 2, 2048, 160, "mxfp4", "mxfp4", "bf16", "f32", "gelu_tanh", "softmax", False),
    (16, 64, 8, 256, 64, "mxfp4", "mxfp4", "bf16", "bf16", "silu", "softmax", False),
    (64, 3, 2, 96, 160, "mxfp4", "mxfp4", "f16", "f32", "silu", "sigmoid", False),
    (40, 1, 1, 288, 96, "mxfp4", "mxfp4", "bf16", "f32", "silu", "softmax", True),
    (33, 130, 16, 64, 32, "mxfp4", "mxfp4", "bf16", "bf16", "silu", "softmax", True),
    (2, 8, 2, 4096, 1024, "affine64.bf16", "affine64.bf16", "bf16", "bf16", "silu", "softmax", True),
    (9, 6, 2, 512, 256, "affine32.f16", "affine128.bf16", "f16", "f32", "gelu_tanh", "softmax", True),
    (20, 3, 2, 256, 512, "q4k", "q4k", "bf16", "f32", "silu", "sigmoid", True),
    (5, 4, 4, 1280, 256, "q4k", "mxfp4", "f16", "f16", "silu", "softmax", False),
    (12, 4, 2, 160, 96, "sym4", "sym4.32", "bf16", "f32", "silu", "softmax", True),
    (6, 300, 5, 128, 64, "affine64.bf16", "sym4", "f16", "f32", "gelu_tanh", "sigmoid", True),
    (1, 2, 2, 256, 24576, "affine32.bf16", "affine32.bf16", "bf16", "f32", "silu", "softmax", True),
    (1, 2, 2, 20480, 64, "affine32.bf16", "mxfp4", "bf16", "f32", "silu", "softmax", True),
    (5, 1, 1, 114656, 32, "mxfp4", "mxfp4", "bf16", "f32", "silu", "softmax", True),
    (5, 1, 1, 32, 114656, "mxfp4", "mxfp4", "f16", "f32", "silu", "softmax", True),
    (6, 1, 1, 44800, 64, "q4k", "mxfp4", "bf16", "f32", "silu", "softmax", True),
    (6, 1, 1, 64, 28640, "mxfp4", "affine32.bf16", "bf16", "f32", "silu", "softmax", True),
    (5, 1, 1, 28640, 32, "affine32.f16", "mxfp4", "f16", "f32", "silu", "softmax", True),
]


@pytest.mark.parametrize("c", CASES, ids=[f"{c[0]}x{c[3]}x{c[4]}-{c[2]}of{c[1]}-{c[5]}-{c[7]}" for c in CASES])
def test_layer(q, c):
    M, E, topk, K, inner, fu, fd, dt, yd, kind, score, norm = c
    print("moe", *c, flush=True)
    rng = np.random.default_rng(M * E + K)
    g, u, n = stack(q, fu, rng, E, inner, K, dt), stack(q, fu, rng, E, inner, K, dt), stack(q, fd, rng, E, K, inner, dt)
    x, x64 = dev(rng.normal(size=(M, K)), dt)
    r, r64 = dev(rng.normal(size=(E, K)) / np.sqrt(K), dt)
    o = q.qmoe_forward(g[0], n[0], x, g[1], u[1], n[1], experts=E, topk=topk, router=r, score=score, norm=norm,
                       act=kind, y_dtype=yd)
    ids, w = moe.route(x64, r64, topk, score, norm)
    assert np.array_equal(o.ids.cpu().numpy(), ids)
    within(o.weights, w, 2.0 ** -23 * w, "weights")
    ref = check(o, x64, ids, f64(o.weights), parts(g), parts(u), parts(n), kind, dt, yd)
    if M <= 3:
        stated = moe.layer(x64, ids, f64(o.weights), g[2], u[2], n[2], kind)
        assert np.allclose(stated, ref, rtol=1e-9, atol=1e-12)
    # the same with the choice given
    p = q.qmoe_forward(g[0], n[0], x, g[1], u[1], n[1], experts=E, topk=topk, ids=o.ids, weights=o.weights,
                       act=kind, y_dtype=yd)
    assert torch.equal(p.y, o.y)
    # a token's result does not depend on the others
    one = q.qmoe_forward(g[0], n[0], x[M - 1:].contiguous(), g[1], u[1], n[1], experts=E, topk=topk, router=r,
                         score=score, norm=norm, act=kind, y_dtype=yd)
    assert torch.equal(one.y[0], o.y[-1]) and torch.equal(one.ids[0], o.ids[-1])


def small(q, seed, M=6, E=5, K=128, inner=96, dt="bf16"):
    rng = np.random.default_rng(seed)
    g, u, n = (stack(q, "mxfp4", rng, E, a, b, dt) for a, b in ((inner, K), (inner, K), (K, inner)))
    x, x64 = dev(rng.normal(size=(M, K)), dt)
    return rng, g, u, n, x, x64


def test_given_choices(q):
    """Ids in any order, the same one twice, none, and ids outside the layer."""
    rng, g, u, n, x, x64 = small(q, 1)
    ids = np.array([[0, 1, 2], [3, 3, 3], [-1, 4, -1], [-1, -1, -1], [5, 99, 2], [1, 4, 1]], np.int32)
    w = rng.normal(size=(6, 3)).astype(np.float32)
    o = q.qmoe_forward(g[0], n[0], x, g[1], u[1], n[1], experts=5, topk=3, ids=torch.from_numpy(ids).cuda(),
                       weights=torch.from_numpy(w).cuda(), y_dtype="f32")
    check(o, x64, ids, w.astype(np.float64), parts(g), parts(u), parts(n), "silu", "bf16", "f32")
    assert not f64(o.y)[3].any()
    none = q.qmoe_forward(g[0], n[0], x, g[1], u[1], n[1], experts=5, topk=1,
                          ids=torch.full((6, 1), -1, dtype=torch.int32, device="cuda"),
                          weights=torch.ones((6, 1), device="cuda"))
    assert not f64(none.y).any()


def test_ties_and_nan_logits(q):
    """Equal logits: the lower expert first.  NaN logits are not taken; where
    numbers run out, ids are -1 with weights 0."""
    _, g, u, n, x, x64 = small(q, 2)
    r = torch.zeros((5, 128), dtype=torch.bfloat16, device="cuda")
    r[3] = r[1] = 0.5
    o = q.qmoe_forward(g[0], n[0], x, g[1], u[1], n[1], experts=5, topk=3, router=r)
    s = x64.sum(1) * 0.5
    for m in range(6):
        assert o.ids[m].tolist() == ([1, 3, 0] if s[m] > 0 else [0, 2, 4])
    r[:] = float("nan")
    r[4] = 1.0
    o = q.qmoe_forward(g[0], n[0], x, g[1], u[1], n[1], experts=5, topk=3, router=r)
    assert o.ids.tolist() == [[4, -1, -1]] * 6 and o.weights.tolist() == [[1.0, 0.0, 0.0]] * 6
    assert torch.isfinite(o.y).all()
    r[4] = float("nan")
    o = q.qmoe_forward(g[0], n[0], x, g[1], u[1], n[1], experts=5, topk=3, router=r, norm=False)
    assert o.ids.tolist() == [[-1, -1, -1]] * 6 and not f64(o.y).any() and not f64(o.weights).any()


def test_large_logits(q):
    """Logits far past exp's range, and a token of infinities: the others keep their results."""
    _, g, u, n, x, x64 = small(q, 3)
    rng = np.random.default_rng(4)
    r, r64 = dev(rng.normal(size=(5, 128)) * 1e4, "bf16")
    for score in ("softmax", "sigmoid"):
        o = q.qmoe_forward(g[0], n[0], x, g[1], u[1], n[1], experts=5, topk=2, router=r, score=score, norm=False)
        with np.errstate(over="ignore"):
            ids, w = moe.route(x64, r64, 2, score, False)
        assert np.array_equal(o.ids.cpu().numpy(), ids)
        within(o.weights, w, 2.0 ** -23 * w + 1e-45, "weights")
    y = x.clone()
    y[2] = float("inf")
    p = q.qmoe_forward(g[0], n[0], y, g[1], u[1], n[1], experts=5, topk=2, router=r, score="sigmoid", norm=False)
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(p.y[keep], o.y[keep]) and torch.equal(p.ids[keep], o.ids[keep])


def test_experts_are_concatenated_layers(q):
    """Experts stacked by qpack_concat_n against the layers one by one."""
    rng = np.random.default_rng(5)
    E, K, inner = 3, 256, 64
    D = q.QDesc
    def quant(d):
        return q.qpack_quantize(d, torch.from_numpy((rng.normal(size=(d.N, d.K)) * 0.1).astype(np.float32)).cuda())
    du, dd = D.mxfp4(inner, K), D.mxfp4(K, inner)
    gs, us, ns = ([quant(d) for _ in range(E)] for d in (du, du, dd))
    (su, g), (_, u), (sd, n) = q.concat_n([du] * E, gs), q.concat_n([du] * E, us), q.concat_n([dd] * E, ns)
    x, _ = dev(rng.normal(size=(4, K)), "bf16")
    ids = torch.tensor([[2, 0]] * 4, dtype=torch.int32, device="cuda")
    w = torch.full((4, 2), 0.5, device="cuda")
    o = q.qmoe_forward(su, sd, x, g, u, n, experts=E, topk=2, ids=ids, weights=w, y_dtype="f32")
    ref = sum(0.5 * q.qlinear_forward(dd, q.qlinear_gated_forward(du, x, gs[e], us[e]).h, ns[e], y_dtype="f32")
              for e in (2, 0))
    assert torch.allclose(o.y, ref, rtol=1e-6, atol=1e-7)


def test_captured_replayed_and_on_two_streams(q):
    rng, g, u, n, x, _ = small(q, 6, M=20, E=9, K=256, inner=160)
    r, _ = dev(rng.normal(size=(9, 256)), "bf16")

    def step(t):
        return q.qmoe_forward(g[0], n[0], q.qnorm_forward(t).y, g[1], u[1], n[1], experts=9, topk=4, router=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x)
    for k in range(4):
        x.copy_(torch.from_numpy(rng.normal(size=x.shape)))
        eager = [t.clone() for t in step(x)]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b), k
    xs = [torch.randn((20, 256), device="cuda").bfloat16() for _ in range(2)]
    want = [step(t) for t in xs]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for i in range(2):
            with torch.cuda.stream(st[i]):
                got.append(step(xs[i]))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for v, w in zip(got, want) for a, b in zip(v, w))


def test_outputs_stay_inside(q):
    """Outputs and the workspace: bytes past their sizes are left as they were."""
    import ctypes
    rng, g, u, n, x, _ = small(q, 7)
    r, _ = dev(rng.normal(size=(5, 128)), "bf16")
    want = q.qmoe_forward(g[0], n[0], x, g[1], u[1], n[1], experts=5, topk=3, router=r)
    size = ctypes.c_size_t(0)
    q._check(q.lib.qmoe_workspace_bytes(g[0]._cref, n[0]._cref, 6, 5, 3, ctypes.byref(size)))
    bufs = [torch.full((k + 1024,), 77, dtype=t, device="cuda") for k, t in
            ((18, torch.int32), (18, torch.float32), (6 * 128, torch.bfloat16), (size.value, torch.uint8))]
    w = [ctypes.byref(q._wstruct(s[1])) for s in (g, u, n)]
    q._run(x.device, q.lib.qmoe_forward, g[0]._cref, n[0]._cref, 5, 3, x.data_ptr(), 1, 6, r.data_ptr(), 0, 1,
           bufs[0].data_ptr(), bufs[1].data_ptr(), *w, 0, bufs[2].data_ptr(), 1, bufs[3].data_ptr(), size.value)
    torch.cuda.synchronize()
    for b, k in zip(bufs, (18, 18, 6 * 128, size.value)):
        assert torch.all(b[k:] == 77)
    assert torch.equal(bufs[2][:6 * 128].view(6, 128), want.y)


def test_binding_refuses_wrong_tensors(q):
    rng, g, u, n, x, _ = small(q, 8)
    r, _ = dev(rng.normal(size=(5, 128)), "bf16")
    ids, w = torch.zeros((6, 2), dtype=torch.int32, device="cuda"), torch.ones((6, 2), device="cuda")

    def call(up=g[0], down=n[0], t=x, gate=g[1], E=5, k=2, **kw):
        return q.qmoe_forward(up, down, t, gate, u[1], n[1], experts=E, topk=k, **(kw or dict(router=r)))
    call()
    for err, kw in ((ValueError, dict(router=r, ids=ids, weights=w)), (ValueError, dict(ids=ids)),
                    (ValueError, dict(weights=w)), (ValueError, dict(router=r[:4])), (TypeError, dict(router=r.half())),
                    (TypeError, dict(ids=ids.long(), weights=w)), (ValueError, dict(ids=ids[:, :1], weights=w)),
                    (ValueError, dict(t=x[:, :64], router=r)), (ValueError, dict(router=r, score="max")),
                    (ValueError, dict(router=r, act="relu")), (ValueError, dict(gate=n[1] | dict(scales=None))),
                    (q.QLinearError, dict(t=x[:0])), (q.QLinearError, dict(k=6)),
                    (q.QLinearError, dict(E=4, router=r[:4].contiguous()))):
        with pytest.raises(err):
            call(**kw)


def routed(q, x, r, topk, score="softmax", norm=True):
    """(ids, weights) of a layer of small experts."""
    _, g, u, n, _, _ = small(q, 2, M=x.shape[0], E=r.shape[0], K=x.shape[1])
    o = q.qmoe_forward(g[0], n[0], x, g[1], u[1], n[1], experts=r.shape[0], topk=topk, router=r, score=score, norm=norm)
    return o.ids.cpu().numpy(), o.weights


@pytest.mark.parametrize("E", [5, 20])       # the router in one kernel, and in two
@pytest.mark.parametrize("up", [70, 100, -70, -90, 0])
def test_router_products_past_fp32(q, E, up):
    """bf16 rows and routers whose products lie outside fp32's range: logits are held
    in fp64, so the choice is the statement's."""
    rng = np.random.default_rng(100 + E + up)
    x, x64 = dev(rng.normal(size=(6, 128)) * 2.0 ** up, "bf16")
    r, r64 = dev(rng.normal(size=(E, 128)) * 2.0 ** up, "bf16")
    for score in ("softmax", "sigmoid"):
        print("router", E, up, score, flush=True)
        with np.errstate(over="ignore"):
            ids, w = moe.route(x64, r64, 4, score, False)
        got, gw = routed(q, x, r, 4, score, False)
        assert np.array_equal(got, ids)
        within(gw, w, 2.0 ** -23 * w + 1e-45, "weights")


@pytest.mark.parametrize("E", [5, 20])
def test_infinite_logits(q, E):
    """A logit of -infinity is a number: taken last, with weight 0.  One of +infinity
    is taken first; a softmax whose largest logit is infinite is NaN, normed or not."""
    rng = np.random.default_rng(E)
    x, _ = dev(np.abs(rng.normal(size=(6, 128))) + 0.1, "bf16")
    r, r64 = dev(rng.normal(size=(E, 128)) / 16, "bf16")
    order = np.argsort(-(f64(x) @ r64.T), axis=1, kind="stable")
    s = r.clone()
    s[2, 0] = -float("inf")
    s[3, 0] = float("nan")
    want = np.array([[e for e in row if e not in (2, 3)] + [2, -1] for row in order])
    if E == 5:
        for score in ("softmax", "sigmoid"):
            for norm in (False, True):
                ids, w = routed(q, x, s, 5, score, norm)
                assert np.array_equal(ids, want)
                w = f64(w)
                assert not w[:, 3:].any() and np.all(w[:, :3] > 0)
                if norm:
                    assert np.allclose(w.sum(1), 1, atol=1e-6)
    s = r.clone()
    s[1, 0] = float("inf")
    for norm in (False, True):
        ids, w = routed(q, x, s, 3, "softmax", norm)
        assert np.all(ids[:, 0] == 1) and np.isnan(f64(w)).all()
        ids, w = routed(q, x, s, 3, "sigmoid", norm)
        w = f64(w)
        assert np.all(ids[:, 0] == 1) and np.isfinite(w).all() and (norm or np.all(w[:, 0] == 1))
    s[:, 0] = -float("inf")
    ids, w = routed(q, x, s, 3, "softmax", True)
    assert np.all(ids == [0, 1, 2]) and np.isnan(f64(w)).all()
    ids, w = routed(q, x, s, 3, "sigmoid", True)
    assert np.all(ids == [0, 1, 2]) and not f64(w).any()
    # NaN weights reach y; the other tokens keep their results
    _, g, u, n, _, _ = small(q, 2, E=5)
    y = x.clone()
    y[4] = float("inf")
    t = r[:5].abs() + 0.01
    a = q.qmoe_forward(g[0], n[0], x, g[1], u[1], n[1], experts=5, topk=2, router=t)
    b = q.qmoe_forward(g[0], n[0], y, g[1], u[1], n[1], experts=5, topk=2, router=t)
    keep = [0, 1, 2, 3, 5]
    assert torch.equal(a.y[keep], b.y[keep]) and torch.isnan(b.weights[4]).all() and torch.isnan(b.y[4]).all()


# ---------------------------------------------------------------- layers with many units of work
MAG = {"bf16": 128.0, "f16": 1024.0}


def big_stack(q, fmt, g, E, rows, K, dt):
    """A stacked layer of random codes: descriptor, buffers, and e -> the expert's weights
    and the magnitudes that its chunks' sums pass through (both fp64, on the GPU)."""
    d = desc(q, fmt, E * rows, K)
    N, cuda = E * rows, dict(device="cuda", generator=g)
    words = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), dtype=torch.int32, **cuda)
    buf = dict(qweight=words, qweight_hi=None, scales=None, zeros=None, steps=None)
    if fmt == "mxfp4":
        buf["scales"] = torch.randint(118, 123, (N, K // 32), dtype=torch.uint8, **cuda)
    elif fmt == "q4k":
        buf["scales"] = torch.randint(1, 64, (N, K // 32), dtype=torch.uint8, **cuda)
        buf["zeros"] = torch.randint(0, 64, (N, K // 32), dtype=torch.uint8, **cuda)
        steps = torch.rand((N, K // 256, 2), **cuda) * torch.tensor([4e-4, 0.2], device="cuda") + 1e-4
        buf["steps"] = steps.half().view(torch.int32).view(N, K // 256)
    elif fmt.startswith("sym4"):
        words |= 0x11111111
        buf["scales"] = torch.rand((N, K // d.group_size), **cuda) * 0.01 + 0.005
    else:
        s = torch.rand((N, K // d.group_size), **cuda) * 0.01 + 0.005
        buf["scales"], buf["zeros"] = s.to(DT[fmt[-4:].strip(".")]), (s * -7).to(DT[fmt[-4:].strip(".")])

    def expert(e):
        b = {k: None if v is None else v[e * rows:(e + 1) * rows] for k, v in buf.items()}
        c = torch.stack([(b["qweight"] >> (4 * i)) & 15 for i in range(8)], -1).view(rows, K).double()
        rep = lambda t, n: t.double().repeat_interleave(n, 1)
        if fmt == "mxfp4":
            m = torch.tensor(list(mx.VALUES) + list(-mx.VALUES), dtype=torch.float64, device="cuda")
            w = m[c.long()] * torch.exp2(rep(b["scales"], 32) - 127)
            return w, w.abs()
        if fmt == "q4k":
            st = b["steps"].contiguous().view(torch.float16).view(rows, K // 256, 2)
            S = rep(b["scales"], 32) * rep(st[..., 0], 256)
            z = S * rep(b["zeros"], 32) * rep(st[..., 1], 256)
            return c * S - z, (2 * MAG[dt] + 32) * S + z.abs()
        S = rep(b["scales"], d.group_size)
        z = 8 * S if fmt.startswith("sym4") else -rep(b["zeros"], d.group_size)
        return c * S - z, (2 * MAG[dt] + 32) * S + z.abs()
    return d, buf, expert


# Sizes at which an expert's rows take several passes, a row all of a wave's steps, and the last
# tile is part of one: M, E, topk, K, inner, formats, dt, act
BIG = [
    (12, 64, 8, 1056, 480, "mxfp4", "mxfp4", "bf16", "silu"),       # a wave per row, 3 steps
    (4, 64, 16, 1056, 480, "mxfp4", "mxfp4", "f16", "gelu_tanh"),   # the same, up to four tokens
    (9, 64, 8, 5152, 416, "mxfp4", "mxfp4", "bf16", "silu"),        # 11 steps, x step by step; five passes down
    (20, 128, 8, 1056, 1056, "mxfp4", "mxfp4", "bf16", "silu"),     # two passes of three steps both ways
    (64, 512, 16, 288, 544, "mxfp4", "mxfp4", "f16", "silu"),       # the limits; four passes up, two of two steps down
    (3, 64, 16, 2848, 544, "mxfp4", "mxfp4", "bf16", "gelu_tanh"),  # two passes down, up to four tokens
    (40, 16, 4, 2080, 4640, "mxfp4", "mxfp4", "bf16", "silu"),      # 10 steps down, step by step
    (60, 12, 4, 1056, 2080, "mxfp4", "mxfp4", "f16", "silu"),       # many tokens each
    (16, 64, 8, 1088, 1088, "affine64.bf16", "affine64.bf16", "bf16", "silu"),
    (4, 64, 16, 1088, 544, "affine32.f16", "affine32.bf16", "f16", "silu"),
    (20, 64, 8, 1280, 2560, "q4k", "q4k", "bf16", "gelu_tanh"),
    (10, 64, 8, 1056, 2112, "sym4", "sym4.32", "f16", "silu"),
]


@pytest.mark.parametrize("c", BIG, ids=[f"{c[0]}x{c[3]}x{c[4]}-{c[2]}of{c[1]}-{c[5]}-{c[7]}" for c in BIG])
def test_layers_of_many_units(q, c):
    M, E, topk, K, inner, fu, fd, dt, kind = c
    print("moe", *c, flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M * K + inner)
    G, Um, Dn = (big_stack(q, f, gen, E, a, b, dt) for f, a, b in ((fu, inner, K), (fu, inner, K), (fd, K, inner)))
    x = (torch.randn((M, K), device="cuda", generator=gen) * 0.25).to(DT[dt])
    ids = torch.stack([torch.randperm(E, device="cuda", generator=gen)[:topk] for _ in range(M)]).int()
    wts = torch.rand((M, topk), device="cuda", generator=gen)
    o = q.qmoe_forward(G[0], Dn[0], x, G[1], Um[1], Dn[1], experts=E, topk=topk, ids=ids, weights=wts, act=kind,
                       y_dtype="f32")
    again = q.qmoe_forward(G[0], Dn[0], x, G[1], Um[1], Dn[1], experts=E, topk=topk, ids=ids, weights=wts, act=kind,
                           y_dtype="f32")
    assert torch.equal(o.y, again.y)

    def tol(v, w, mag):
        n = w.shape[1]
        return 72 * 2.0 ** -24 * (v @ mag.t()) + 2 * (n // 32 + 24) * 2.0 ** -24 * (v @ w.abs().t())
    x64, ref, lim = x.double(), torch.zeros((M, K), device="cuda").double(), torch.zeros((M, K), device="cuda").double()
    for e in range(E):
        m, slot = (ids == e).nonzero(as_tuple=True)
        if not len(m):
            continue
        (gw, gm), (uw, um), (dw, dm) = G[2](e), Um[2](e), Dn[2](e)
        v = x64[m]
        g, u = v @ gw.t(), v @ uw.t()
        dg, du = tol(v.abs(), gw, gm), tol(v.abs(), uw, um)
        a = torch.from_numpy(mlp.act(g.cpu().numpy(), kind)[0]).cuda()
        h = a * u
        dh = 1.13 * dg * (u.abs() + du) + a.abs() * du + (U[dt] + 2.0 ** -17) * h.abs() + TINY[dt]
        w = wts[m, slot].double()[:, None]
        ref.index_add_(0, m, w * (h @ dw.t()))
        lim.index_add_(0, m, w * (dh @ dw.abs().t() + tol(h.abs() + dh, dw, dm) + 2.0 ** -22 * (h.abs() @ dw.abs().t())))
    err, lim = (o.y.double() - ref).abs(), lim * (1 + 2.0 ** -23) + 2.0 ** -20 * ref.abs() + TINY["f32"]
    assert bool(torch.isfinite(o.y).all()) and bool((err <= lim).all()), float((err / lim).max())
