"""GPU parity of the MLP-block operators with their fp64 statements.

Tolerances.  A value rounded to a 16-bit type is off by at most u times its
size (u = finfo.eps / 2), plus half the smallest subnormal; an fp32 operation
by 2^-24.  Products of two 16-bit values are exact in fp32.  The packed
products are held to the layer's own contract: per element 1e-2 ||x|| max|w|
/ sqrt(K), and relative L2 2e-3; input gradients to what the roundings of
their operands can add up to, and the same relative L2.
"""
import numpy as np
import pytest

import oracle
from helpers import buf_to_np, qformat_of
from oracle import mlp

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -9 * 2, "f16": 2.0 ** -11, "f32": 2.0 ** -24}    # eps / 2
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_weight_only_qlinear_amd import qlinear
    return qlinear


def f64(t):
    return t.detach().double().cpu().numpy()


def dev(a, dt):
    """fp64 array -> device tensor of type dt, and the values it holds."""
    t = torch.from_numpy(np.asarray(a)).to(DT[dt]).cuda()
    return t, f64(t)


def within(got, ref, tol, what):
    err = np.abs(f64(got) - ref)
    assert err.shape == np.broadcast(ref, tol).shape and np.all(np.isfinite(err)), what
    bad = err > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.max(err / (tol + 1e-300)):.3f}x"


def stream_of(rng, M, K):
    x = rng.normal(size=(M, K))
    x[:, rng.integers(0, K)] *= 12.0
    return x


NORM_SIZES = [(1, 1), (3, 7), (1, 64), (5, 8), (2, 512), (9, 520), (4, 2048), (2, 2056), (1, 4096),
              (7, 5121), (2, 8192), (3, 8200), (1, 16384), (2, 32768), (1, 32776), (515, 96)]


# ---------------------------------------------------------------- norm
@pytest.mark.parametrize("M,K", NORM_SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_norm_forward(q, M, K, dt):
    print("norm", M, K, dt, flush=True)
    rng = np.random.default_rng(K)
    x, x64 = dev(stream_of(rng, M, K), dt)
    r, r64 = dev(rng.normal(size=(M, K)), dt)
    w, w64 = dev(1 + 0.2 * rng.normal(size=K), dt)
    eps = 1e-5
    for res, wt in ((None, None), (None, w), (r, w)):
        o = q.qnorm_forward(x, wt, residual=res, eps=eps, need_rstd=True)
        s64 = x64 if res is None else f64(torch.from_numpy(x64 + r64).to(DT[dt]))
        assert np.array_equal(f64(o.s), s64)      # one rounding of the exact sum
        ref = mlp.norm(s64, 1.0 if wt is None else w64, eps)
        # rstd to fp32, its product: 2^-24 each; then the type
        within(o.y, ref, (U[dt] + 2.0 ** -22) * np.abs(ref) + TINY[dt], "y")
        within(o.rstd, mlp.rstd(s64, eps)[:, 0], 2.0 ** -23 * mlp.rstd(s64, eps)[:, 0], "rstd")
        p = q.qnorm_forward(x, wt, residual=res, eps=eps, quantize=True)
        assert p.y is None and np.array_equal(f64(p.s), s64)
        _, ys = mlp.row_codes(ref)
        within(p.ys, ys.astype(np.float64), 2.0 ** -23 * ys, "ys")
        step = f64(p.ys)[:, None]
        # nearest code of the exact value under the stored scale (1e-9: fp64
        # rounding of values up to 127 steps; the clamp at 127 costs nothing,
        # since fl32(max / 127) * 127 >= max (1 - 2^-24) - half a step is far)
        assert np.all(np.abs(ref - f64(p.yq) * step) <= (0.5 + 1e-9) * step)


def test_norm_in_place_and_zero_rows(q):
    rng = np.random.default_rng(5)
    for K in (256, 250):          # the register form and the general one
        x, x64 = dev(rng.normal(size=(6, K)), "bf16")
        r, r64 = dev(rng.normal(size=(6, K)), "bf16")
        x[2] = 0
        r[2] = 0
        ref = q.qnorm_forward(x, residual=r)
        for alias in ("x", "r"):
            xx, rr = x.clone(), r.clone()
            o = q.qnorm_forward(xx, residual=rr, s_out=xx if alias == "x" else rr)
            assert torch.equal(o.s, ref.s) and torch.equal(o.y, ref.y)
            assert torch.equal(rr if alias == "x" else xx, r if alias == "x" else x)
        assert not f64(ref.y)[2].any()
        p = q.qnorm_forward(x, residual=r, quantize=True)
        assert not f64(p.yq)[2].any() and f64(p.ys)[2] == 0


def test_norm_large_values_do_not_overflow(q):
    """bf16 values whose squares pass fp32's range."""
    x, x64 = dev(np.array([[1e30, -2e30, 3e30, 0.0] * 4, [1e-30] * 16]), "bf16")
    ref = mlp.norm(x64, 1.0, 1e-6)
    within(q.qnorm_forward(x).y, ref, (U["bf16"] + 2.0 ** -22) * np.abs(ref), "y")


@pytest.mark.parametrize("M,K", NORM_SIZES + [(1100, 200), (600, 77)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("saved", [False, True])
def test_norm_backward(q, M, K, dt, saved):
    print("norm backward", M, K, dt, saved, flush=True)
    rng = np.random.default_rng(K + 1)
    s, s64 = dev(stream_of(rng, M, K), dt)
    dy, dy64 = dev(rng.normal(size=(M, K)) * 0.1, dt)
    w, w64 = dev(1 + 0.2 * rng.normal(size=K), dt)
    di, di64 = dev(rng.normal(size=(M, K)) * 0.1, dt)
    ck = None
    if saved:
        ck = q.qpack_checkpoint(s)
        s64 = mlp.restore(ck[0].cpu().numpy(), ck[1].cpu().numpy())
    r = torch.from_numpy(mlp.rstd(s64, 1e-5)[:, 0]).float().cuda()
    r64 = f64(r)[:, None]
    for wt, add in ((w, di), (None, None)):
        W, D = (w64, di64) if add is not None else (np.ones(K), 0.0)
        ds, dw = q.qnorm_backward(dy, None if saved else s, r, wt, saved=ck, ds_in=add)
        ref, refw = mlp.norm_backward(dy64, s64, W, r64, D)
        g, xh = np.abs(dy64 * W), np.abs(s64 * r64)
        # up to 8 fp32 operations on each of the three terms, 16 on the mean's
        mag = r64 * (g + xh * np.mean(g * xh, axis=1, keepdims=True)) + np.abs(D)
        within(ds, ref, U[dt] * np.abs(ref) + 2.0 ** -20 * mag + TINY[dt], "ds")
        # fp32 sums of ceil(M / 512) rows, three roundings each, then fp64
        rows = -(-M // min(M, 512)) + 4
        within(dw, refw, rows * 2.0 ** -24 * np.sum(np.abs(dy64) * xh, axis=0) + 1e-38, "dweight")
    only, none = q.qnorm_backward(dy, None if saved else s, r, w, saved=ck, need_dweight=False)
    assert none is None
    none, dw2 = q.qnorm_backward(dy, None if saved else s, r, w, saved=ck, need_ds=False)
    assert none is None
    a, b = q.qnorm_backward(dy, None if saved else s, r, w, saved=ck)
    assert torch.equal(a, only) and torch.equal(b, dw2)


@pytest.mark.parametrize("K", [512, 515, 40960])
@pytest.mark.parametrize("alias", ["dy", "ds_in"])
def test_norm_backward_in_place(q, K, alias):
    """ds written over dy or ds_in (the C call takes the output's address)."""
    rng = np.random.default_rng(K)
    M = 9
    s, dy, di = (dev(rng.normal(size=(M, K)), "bf16")[0] for _ in range(3))
    w, r = dev(rng.normal(size=K), "bf16")[0], torch.rand(M, device="cuda") + 0.5
    ds, dw = q.qnorm_backward(dy, s, r, w, ds_in=di)
    out = dy if alias == "dy" else di
    dw2 = torch.empty_like(dw)
    ws = torch.empty(M * K * 4, dtype=torch.uint8, device="cuda")
    q._check(q.lib.qnorm_backward(dy.data_ptr(), s.data_ptr(), None, None, 1, M, K, w.data_ptr(),
                                  r.data_ptr(), di.data_ptr(), out.data_ptr(), dw2.data_ptr(),
                                  ws.data_ptr(), ws.numel(), q._stream()))
    assert torch.equal(out, ds) and torch.equal(dw2, dw)


# ---------------------------------------------------------------- checkpoints
@pytest.mark.parametrize("M,K", [(1, 1), (2, 63), (3, 64), (5, 65), (1, 72), (4, 128), (19, 1000),
                                 (33, 4099), (7, 14336)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_checkpoint(q, M, K, dt):
    print("checkpoint", M, K, dt, flush=True)
    rng = np.random.default_rng(M * K)
    x, x64 = dev(stream_of(rng, M, K), dt)
    x[M // 2] = 0
    x64[M // 2] = 0
    codes, scales = q.qpack_checkpoint(x)
    rq, rs = mlp.checkpoint(x64)
    assert np.array_equal(codes.cpu().numpy(), rq) and np.array_equal(scales.cpu().numpy(), rs)
    for od in ("f32", "bf16", "f16"):
        got = q.qpack_checkpoint_restore((codes, scales), od)
        ref = torch.from_numpy(mlp.restore(rq, rs)).float().to(DT[od])   # one fp32 product
        assert torch.equal(got.cpu(), ref), od


def test_checkpoint_scales_over_the_range(q):
    """Groups of very small and very large values, subnormal scales and
    quotients among them."""
    rng = np.random.default_rng(9)
    v = rng.normal(size=(130, 64)) * 10.0 ** rng.uniform(-39, 38, size=(130, 1))
    v[0] = 0
    v[1, 1:] = 0
    for K in (64, 60):
        x, x64 = dev(np.clip(v[:, :K], -3e38, 3e38), "bf16")
        codes, scales = q.qpack_checkpoint(x)
        rq, rs = mlp.checkpoint(x64)
        assert np.array_equal(scales.cpu().numpy(), rs)
        assert np.array_equal(codes.cpu().numpy(), rq)


def test_checkpoint_ties_go_to_even(q):
    """Scales 3 and 2 with values half way between codes."""
    x = torch.zeros((2, 64), dtype=torch.float16)
    x[0, :5] = torch.tensor([381.0, 7.5, -7.5, 4.5, 1.5])      # 2.5, -2.5, 1.5, 0.5 steps of 3
    x[1, :4] = torch.tensor([254.0, 5.0, 3.0, -1.0])
    codes, scales = q.qpack_checkpoint(x.cuda())
    assert scales.cpu()[:, 0].tolist() == [3.0, 2.0]
    assert codes.cpu()[0, :5].tolist() == [127, 2, -2, 2, 0]
    assert codes.cpu()[1, :4].tolist() == [127, 2, 2, 0]


# ---------------------------------------------------------------- packed products
def formats(q, N, K):
    D = q.QDesc
    out = [D.affine(N, K, 4, 32, "bf16"), D.sym4(N, K), D.sym4(N, K, 32)]
    if K % 64 == 0:
        out += [D.affine(N, K, 2, 64, "f16"), D.affine(N, K, 4, 64, "bf16"), D.affine(N, K, 8, 64, "bf16"),
                D.affine(N, K, 8, 32, "f16"), D.affine(N, K, 2, 32, "bf16")]
    if K % 128 == 0:
        out += [D.affine(N, K, 4, 128, "f16"), D.sym4(N, K, 128), D.affine(N, K, 2, 128, "bf16")]
    if K % 256 == 0:
        out += [D.q4k(N, K), D.q6k(N, K)]
    return out


def packed(q, d, rng, scale=0.05):
    """A layer's buffers and its dequantized fp64 matrix."""
    W = (rng.normal(size=(d.N, d.K)) * scale).astype(np.float32)
    buf = q.qpack_quantize(d, torch.from_numpy(W).cuda())
    f = qformat_of(d)
    w64 = oracle.dequant_f64(oracle.quantize(W, f), f)
    return buf, w64


def rel_limit(ref, od, rel):
    """Relative L2 allowed: `rel`, and what rounding to the type costs."""
    if od == "f32":
        return rel
    r = f64(torch.from_numpy(ref).to(DT[od]))
    return rel + oracle.rel_l2(r, ref)


def product_tolerance(D, w):
    """Largest error of a product of D [M, n] and w [n, K] whose operands are
    rounded to fp16.  D once: 2^-11 of each value, and for the smallest half
    a subnormal, 2^-25 of a row scaled into [2^14, 2^15): 2^-39 of its
    maximum.  A weight at most twice at its own size (2 * 2^-11; Q4K adds two
    rounded parts, the others round once), the second part of a split scale or
    offset once more at 2^-11 of a 2^-11 part of up to 2 max|w|: 2^-21 max|w|,
    taken double.  The sums: n + 32 additions of 2^-24.  (The layer's contract
    for exact activations, 1e-2 ||x|| max|w| / sqrt(n), has no room for D's own
    rounding: at n = 2000 it allows 2.2e-4, under half of one 2^-11.)"""
    a, v = np.abs(D), np.abs(w)
    n = w.shape[0]
    return (2.0 ** -11 + 2.0 ** -10 + 2.0 ** -20 + (n + 32) * 2.0 ** -24) * (a @ v) + \
        2.0 ** -20 * v.max() * a.sum(axis=1, keepdims=True) + \
        2.0 ** -39 * a.max(axis=1, keepdims=True) * v.sum(axis=0)


GATED_SIZES = [(1, 48, 512), (1, 1, 256), (3, 100, 256), (8, 64, 768), (16, 257, 512), (17, 130, 512),
               (70, 64, 256), (300, 200, 512), (5, 96, 96), (40, 33, 160), (2, 65, 320), (33, 448, 320),
               (1, 300, 4096), (1, 33, 5120), (1, 70, 8192), (1, 37, 16384), (1, 90, 1056), (6, 35, 4096),
               (2, 33, 4096), (2, 50, 8192), (2, 40, 512), (1, 20, 65536), (4, 20, 65536), (2, 31, 2560),
               (2, 37, 5120), (16, 41, 2176)]


# enough tiles for whole rounds, a last round in halves, and halves alone
LARGE = [(1000, 6000, 256), (1500, 8000, 256), (700, 5000, 256), (700, 5006, 256)]


@pytest.mark.parametrize("M,N,K", GATED_SIZES + LARGE)
@pytest.mark.parametrize("save", [False, True])
def test_gated_forward(q, M, N, K, save):
    rng = np.random.default_rng(M + N)
    for i, d in enumerate(formats(q, N, K)):
        if (M, N, K) in LARGE and (d.fmt, d.group_size) not in (("affine", 64), ("sym4", K), ("q6k", 16)):
            continue
        dt, kind = ("bf16", "f16")[i % 2], ("silu", "gelu_tanh")[(i // 2) % 2]
        hd = (dt, "f32")[i % 3 == 2]
        print("gated", M, N, K, d.fmt, d.bits, d.group_size, dt, hd, kind, save, flush=True)
        (bg, wg), (bu, wu) = packed(q, d, rng), packed(q, d, rng)
        x, x64 = dev(rng.normal(size=(M, K)), dt)
        c1, c164 = dev(rng.normal(size=N) * 0.3, dt)
        c2, c264 = dev(rng.normal(size=N) * 0.3, dt)
        biased = i % 2 == 0
        o = q.qlinear_gated_forward(d, x, bg, bu, act=kind, bias_gate=c1 if biased else None,
                                    bias_up=c2 if biased else None, h_dtype=hd, save=save)
        g, u, h = mlp.gated(x64, wg, wu, c164 if biased else 0.0, c264 if biased else 0.0, kind)
        # exact codes: the layer's contract; staged: fp16 weights, whose
        # rounding alone (1.4e-4 rms of each weight) comes to 0.4 of that
        # contract's 1e-2 max|w| / sqrt(K) at K = 8192, so it is bounded by
        # what the roundings can add up to
        staged = save or M > 16 or (M > 1 and K % 128 != 0)
        dg, du = (product_tolerance(x64, v.T) if staged else oracle.maxabs_bound(x64, np.abs(v).max(), K)
                  for v in (wg, wu))
        dg, du = dg + 2.0 ** -22 * np.abs(g), du + 2.0 ** -22 * np.abs(u)
        # |act'| <= 1.13; the fp32 logistic's argument and exponential: 2^-17
        tol = 1.13 * dg * (np.abs(u) + du) + np.abs(mlp.act(g, kind)[0]) * du + \
            (U[hd] + 2.0 ** -17) * np.abs(h) + TINY[hd]
        within(o.h, h, tol, "h")
        # first order: g and u are each within 2e-3 of themselves, as L2 over
        # many outputs (one output alone has no relative bound: |g| may be any
        # part of the sum |x| |w| of which the weights' rounding takes 2^-11)
        if h.size >= 256:
            assert oracle.rel_l2(f64(o.h), h) <= rel_limit(h, hd, 6e-3)
        assert (o.gate is None) == (not save)
        if save:
            for (codes, sc), v, e in ((o.gate, g, dg), (o.up, u, du)):
                got = mlp.restore(codes.cpu().numpy(), sc.cpu().numpy())
                step = np.repeat(f64(sc), 64, axis=1)[:, :N]
                assert np.all(np.abs(got - v) <= (0.5 + 1e-4) * step + e)
                top = mlp.checkpoint(v)[1].astype(np.float64)
                m = np.pad(e, ((0, 0), (0, -N % 64))).reshape(M, -1, 64).max(-1) / 127
                assert np.all(np.abs(f64(sc) - top) <= m + 2.0 ** -22 * top)


def test_gated_is_the_pair_of_layers(q):
    """The same layers through qlinear_forward and torch's product."""
    rng = np.random.default_rng(3)
    d = q.QDesc.affine(320, 512, 4, 64, "bf16")
    (bg, _), (bu, _) = packed(q, d, rng), packed(q, d, rng)
    for M in (4, 64):
        x, _ = dev(rng.normal(size=(M, 512)), "bf16")
        g = q.qlinear_forward(d, x, bg, y_dtype="f32")
        u = q.qlinear_forward(d, x, bu, y_dtype="f32")
        ref = f64(torch.nn.functional.silu(g) * u)
        got = f64(q.qlinear_gated_forward(d, x, bg, bu, h_dtype="f32").h)
        assert oracle.rel_l2(got, ref) <= 4e-3


def test_gated_wide_range_bf16(q):
    """bf16 rows past fp16's range, and rows of zeros."""
    rng = np.random.default_rng(4)
    d = q.QDesc.affine(64, 256, 4, 64, "bf16")
    (bg, wg), (bu, wu) = packed(q, d, rng), packed(q, d, rng)
    for M in (3, 20):
        v = rng.normal(size=(M, 256))
        v[0] *= 1e6
        v[1] = 0
        v[2] *= 1e-6
        x, x64 = dev(v, "bf16")
        g, u, h = mlp.gated(x64, wg, wu, 0.0, 0.0, "silu")
        got = f64(q.qlinear_gated_forward(d, x, bg, bu, h_dtype="f32").h)
        assert not got[1].any()
        for m in (0, 2):
            assert oracle.rel_l2(got[m], h[m]) <= 6e-3


BWD_SIZES = [(1, 48, 256), (3, 100, 512), (17, 1, 256), (64, 63, 320), (70, 130, 768), (130, 257, 512),
             (300, 192, 96), (5, 1000, 160), (129, 70, 1024), (260, 640, 320)]


@pytest.mark.parametrize("M,N,K", BWD_SIZES)
def test_linear_backward(q, M, N, K):
    rng = np.random.default_rng(N + K)
    for i, d in enumerate(formats(q, N, K)):
        dt = ("bf16", "f16")[i % 2]
        xd = (dt, "f32")[i % 3 == 1]
        print("linear backward", M, N, K, d.fmt, d.bits, d.group_size, dt, xd, flush=True)
        buf, w64 = packed(q, d, rng)
        dy, dy64 = dev(rng.normal(size=(M, N)) * 1e-2, dt)
        if M > 2:
            dy[1] = 0
            dy64[1] = 0
        got = q.qlinear_backward(d, dy, buf, dx_dtype=xd)
        ref = dy64 @ w64
        tol = product_tolerance(dy64, w64) * (1 + U[xd]) + U[xd] * np.abs(ref) + TINY[xd]
        within(got, ref, tol, "dx")
        assert oracle.rel_l2(f64(got), ref) <= rel_limit(ref, xd, 2e-3)


@pytest.mark.parametrize("M,N,K", BWD_SIZES)
def test_gated_backward(q, M, N, K):
    rng = np.random.default_rng(N * K)
    for i, d in enumerate(formats(q, N, K)):
        dt, kind = ("bf16", "f16")[i % 2], ("silu", "gelu_tanh")[(i // 2) % 2]
        xd = (dt, "f32")[i % 3 == 1]
        print("gated backward", M, N, K, d.fmt, d.bits, d.group_size, dt, xd, kind, flush=True)
        (bg, wg), (bu, wu) = packed(q, d, rng), packed(q, d, rng)
        dh, dh64 = dev(rng.normal(size=(M, N)) * 1e-2, dt)
        ck = []
        for k in range(2):
            c, s = mlp.checkpoint(rng.normal(size=(M, N)) * 2)
            ck.append((c, s, torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()))
        g, u = (mlp.restore(c[0], c[1]) for c in ck)
        o = q.qlinear_gated_backward(d, dh, bg, bu, ck[0][2:], ck[1][2:], act=kind, dx_dtype=xd)
        dx, rg, ru = mlp.gated_backward(dh64, g, u, wg, wu, kind)
        # fp32 chains of fewer than 16 operations around one exponential
        e = 2.0 ** -17
        within(o.dgate, rg, U[dt] * np.abs(rg) + e * np.abs(dh64 * u) * (1 + np.abs(g)) + TINY[dt], "dgate")
        within(o.dup, ru, U[dt] * np.abs(ru) + e * np.abs(dh64) * (1 + np.abs(g)) + TINY[dt], "dup")
        both = np.concatenate([rg, ru], axis=1)
        # dg and du themselves: the fp32 chains above
        own = e * (np.abs(dh64 * u) * (1 + np.abs(g)) @ np.abs(wg) +
                   np.abs(dh64) * (1 + np.abs(g)) @ np.abs(wu))
        tol = (product_tolerance(both, np.concatenate([wg, wu])) + own) * (1 + U[xd]) + \
            U[xd] * np.abs(dx) + TINY[xd]
        within(o.dx, dx, tol, "dx")
        assert oracle.rel_l2(f64(o.dx), dx) <= rel_limit(dx, xd, 2e-3)
        p = q.qlinear_gated_backward(d, dh, bg, bu, ck[0][2:], ck[1][2:], act=kind, dx_dtype=xd,
                                     need_dpre=False)
        assert p.dgate is None and torch.equal(p.dx, o.dx)


# ---------------------------------------------------------------- together
def _block(q, rng, M, K, N, dt="bf16"):
    d, dn = q.QDesc.affine(N, K, 4, 64, "bf16"), q.QDesc.q4k(K, N)
    (g, wg), (u, wu), (n, wn) = packed(q, d, rng), packed(q, d, rng), packed(q, dn, rng)
    x, x64 = dev(rng.normal(size=(M, K)), dt)
    r, r64 = dev(rng.normal(size=(M, K)), dt)
    w, w64 = dev(1 + 0.1 * rng.normal(size=K), dt)
    return d, dn, (g, u, n), (wg, wu, wn), (x, r, w), (x64, r64, w64)


def test_mlp_block_training_step(q):
    """Norm, gated pair, down projection, and back: the gradients against the
    fp64 chain."""
    rng = np.random.default_rng(11)
    M, K, N, eps = 96, 512, 768, 1e-5
    d, dn, (bg, bu, bn), (wg, wu, wn), (x, r, w), (x64, r64, w64) = _block(q, rng, M, K, N)
    dy, dy64 = dev(rng.normal(size=(M, K)) * 1e-2, "bf16")
    o = q.qnorm_forward(x, w, residual=r, eps=eps, need_rstd=True)
    f = q.qlinear_gated_forward(d, o.y, bg, bu, save=True)
    y = q.qlinear_forward(dn, f.h, bn)
    dh = q.qlinear_backward(dn, dy, bn)
    gb = q.qlinear_gated_backward(d, dh, bg, bu, f.gate, f.up)
    ds, dw = q.qnorm_backward(gb.dx, o.s, o.rstd, w, ds_in=dy)
    s64 = f64(o.s)
    n64 = mlp.norm(s64, w64, eps)
    g, u, h = mlp.gated(n64, wg, wu, 0.0, 0.0, "silu")
    assert oracle.rel_l2(f64(y), h @ wn.T) <= 1.5e-2      # four bf16 roundings of 2^-8 at most
    rdh = dy64 @ wn
    rdx, _, _ = mlp.gated_backward(rdh, g, u, wg, wu, "silu")
    rds, rdw = mlp.norm_backward(rdx, s64, w64, mlp.rstd(s64, eps), dy64)
    # the checkpoints' half code steps (about 0.6 % of g and u each) and bf16
    assert oracle.rel_l2(f64(gb.dx), rdx) <= 2.5e-2
    assert oracle.rel_l2(f64(ds), rds) <= 2.5e-2
    assert oracle.rel_l2(f64(dw), rdw) <= 2.5e-2


def test_norm_feeds_a8w4(q):
    """Decode on int8 rows: the norm's codes straight into the a8w4 product."""
    rng = np.random.default_rng(12)
    d = q.QDesc.sym4(200, 512)
    buf, w64 = packed(q, d, rng)
    x, _ = dev(rng.normal(size=(3, 512)), "bf16")
    r, _ = dev(rng.normal(size=(3, 512)), "bf16")
    o = q.qnorm_forward(x, residual=r, quantize=True)
    y = q.qlinear_forward_a8w4(d, o.yq, o.ys, buf, y_dtype="f32")
    ref = (f64(o.yq) * f64(o.ys)[:, None]) @ w64.T
    within(y, ref, 2.0 ** -23 * np.abs(ref) + 1e-30, "y")


def test_block_captured_and_replayed(q):
    """Forward and backward captured into one graph, replayed on new inputs
    with eager work between: every replay equals the eager result."""
    rng = np.random.default_rng(13)
    M, K, N = 40, 256, 320
    d, dn, (bg, bu, bn), _, (x, r, w), _ = _block(q, rng, M, K, N - 64)
    dy = torch.zeros_like(x)

    def step():
        o = q.qnorm_forward(x, w, residual=r, need_rstd=True)
        f = q.qlinear_gated_forward(d, o.y, bg, bu, save=True)
        dh = q.qlinear_backward(dn, dy, bn)
        gb = q.qlinear_gated_backward(d, dh, bg, bu, f.gate, f.up)
        ds, dw = q.qnorm_backward(gb.dx, o.s, o.rstd, w, ds_in=dy)
        p = q.qnorm_forward(x, w, residual=r, quantize=True)
        c = q.qpack_checkpoint_restore(q.qpack_checkpoint(f.h))
        return [f.h, dh, gb.dx, gb.dgate, gb.dup, ds, dw, p.yq, p.ys, c]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(4):
        for t in (x, r, dy):
            t.copy_(torch.from_numpy(rng.normal(size=t.shape)))
        eager = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, eager)):
            assert torch.equal(a, b), (k, i)


def test_two_streams(q):
    """Two calls at once, each on a stream of its own."""
    rng = np.random.default_rng(14)
    d, dn, (bg, bu, bn), _, (x, r, w), _ = _block(q, rng, 64, 512, 768)
    dy = torch.randn((2, 64, 512), device="cuda").bfloat16()
    want = [q.qlinear_backward(dn, dy[i], bn) for i in range(2)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for i in range(2):
            with torch.cuda.stream(st[i]):
                got.append(q.qlinear_backward(dn, dy[i], bn))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_outputs_stay_inside(q):
    """Bytes past the last row are left as they were."""
    import ctypes
    rng = np.random.default_rng(15)
    M, N, K = 19, 70, 320
    d = q.QDesc.affine(N, K, 4, 64, "bf16")
    (bg, _), (bu, _) = packed(q, d, rng), packed(q, d, rng)
    x = torch.randn((M, K), device="cuda").bfloat16()
    dh = torch.randn((M, N), device="cuda").bfloat16()

    def guarded(rows, cols, dt):
        t = torch.full((rows * cols + 4096,), 77, dtype=dt, device="cuda")
        return t, rows * cols

    outs = {k: guarded(M, c, t) for k, c, t in (
        ("h", N, torch.bfloat16), ("gc", N, torch.int8), ("gs", 2, torch.float32), ("uc", N, torch.int8),
        ("us", 2, torch.float32), ("dg", N, torch.bfloat16), ("du", N, torch.bfloat16),
        ("dx", K, torch.bfloat16))}
    p = {k: v[0].data_ptr() for k, v in outs.items()}
    size = ctypes.c_size_t(0)
    q._check(q.lib.qlinear_backward_workspace_bytes(ctypes.byref(d.c()), M, 1, ctypes.byref(size)))
    ws, n = guarded(1, (size.value + 15) // 16 * 16, torch.uint8)
    fsize = ctypes.c_size_t(0)
    q._check(q.lib.qlinear_gated_workspace_bytes(ctypes.byref(d.c()), M, 1, ctypes.byref(fsize)))
    fws, fn = guarded(1, (fsize.value + 15) // 16 * 16, torch.uint8)
    wg, wu = q._wstruct(bg), q._wstruct(bu)
    q._check(q.lib.qlinear_gated_forward(ctypes.byref(d.c()), x.data_ptr(), 1, M, ctypes.byref(wg),
                                         ctypes.byref(wu), None, None, 0, p["h"], 1, p["gc"], p["gs"],
                                         p["uc"], p["us"], fws.data_ptr(), fsize.value, None))
    q._check(q.lib.qlinear_gated_backward(ctypes.byref(d.c()), dh.data_ptr(), 1, M, ctypes.byref(wg),
                                          ctypes.byref(wu), 0, p["gc"], p["gs"], p["uc"], p["us"],
                                          p["dg"], p["du"], p["dx"], 1, ws.data_ptr(), size.value, None))
    torch.cuda.synchronize()
    for k, (t, used) in dict(outs, ws=(ws, n), fws=(fws, fn)).items():
        assert torch.all(t[used:] == 77), k
    assert torch.equal(outs["h"][0][:M * N].view(M, N),
                       q.qlinear_gated_forward(d, x, bg, bu, save=True).h)


def test_offsets_past_32_bits(q):
    """Matrices of more than 2^32 elements or bytes: their last rows against
    the same rows alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    M, K = 66000, 65536
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    x[:] = torch.randn((1, K), device="cuda", generator=g)
    x[-8:] = torch.randn((8, K), device="cuda", generator=g)
    codes, scales = q.qpack_checkpoint(x)
    c8, s8 = q.qpack_checkpoint(x[-8:].contiguous())
    assert torch.equal(codes[-8:], c8) and torch.equal(scales[-8:], s8)
    y = q.qpack_checkpoint_restore((codes, scales))
    assert torch.equal(y[-8:], q.qpack_checkpoint_restore((c8, s8)))
    assert torch.equal(codes[0], codes[M // 2]) and torch.equal(y[1], y[M // 2])
    del codes, scales, y
    o, t = q.qnorm_forward(x, need_rstd=True), q.qnorm_forward(x[-8:].contiguous(), need_rstd=True)
    assert torch.equal(o.y[-8:], t.y) and torch.equal(o.rstd[-8:], t.rstd)
    ds, _ = q.qnorm_backward(o.y, x, o.rstd, need_dweight=False)
    d8, _ = q.qnorm_backward(t.y, x[-8:].contiguous(), t.rstd, need_dweight=False)
    assert torch.equal(ds[-8:], d8)
    del o, ds, x
    M, N, K = 140000, 16384, 128
    d = q.QDesc.affine(N, K, 4, 64, "bf16")
    w = [q.qpack_quantize(d, torch.randn((N, K), device="cuda", generator=g) * 0.1) for _ in range(2)]
    x = torch.randn((M, K), device="cuda", generator=g).bfloat16()
    f = q.qlinear_gated_forward(d, x, *w, save=True)
    e = q.qlinear_gated_forward(d, x[-300:].contiguous(), *w, save=True)
    # other tiles, another order of the fp32 sums: a bf16 step at most
    assert oracle.rel_l2(f64(f.h[-300:]), f64(e.h)) <= 2.0 ** -8
    assert oracle.rel_l2(f64(f.up[0][-300:]), f64(e.up[0])) <= 2.0 ** -8
    b = q.qlinear_gated_backward(d, f.h, *w, f.gate, f.up)
    tail = [tuple(v[-300:].contiguous() for v in ck) for ck in (f.gate, f.up)]
    c = q.qlinear_gated_backward(d, f.h[-300:].contiguous(), *w, *tail)
    assert torch.equal(b.dgate[-300:], c.dgate) and torch.equal(b.dup[-300:], c.dup)
    assert oracle.rel_l2(f64(b.dx[-300:]), f64(c.dx)) <= 2.0 ** -8


def test_binding_refuses_wrong_tensors(q):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    d = q.QDesc.affine(32, 64, 4, 64)
    w = q.qpack_quantize(d, torch.zeros((32, 64), device="cuda"))
    small = q.qpack_quantize(q.QDesc.affine(16, 64, 4, 64), torch.zeros((16, 64), device="cuda"))
    r = torch.ones(4, device="cuda")
    ok = q.qpack_checkpoint(torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda"))
    dh = torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")
    for err, call in (
            (TypeError, lambda: q.qnorm_forward(x.float())),
            (TypeError, lambda: q.qnorm_forward(x, x[0].half())),
            (ValueError, lambda: q.qnorm_forward(x.t())),
            (ValueError, lambda: q.qnorm_forward(x[:, ::2])),
            (ValueError, lambda: q.qnorm_forward(x, residual=x[:2])),
            (ValueError, lambda: q.qnorm_forward(x, x[0].cpu())),
            (ValueError, lambda: q.qnorm_forward(x, s_out=x)),
            (q.QLinearError, lambda: q.qnorm_forward(x[:0])),
            (q.QLinearError, lambda: q.qnorm_forward(x, eps=0.0)),
            (TypeError, lambda: q.qnorm_backward(x, x, r.double())),
            (ValueError, lambda: q.qnorm_backward(x, x, r, saved=ok)),
            (ValueError, lambda: q.qnorm_backward(x, None, r, saved=ok)),
            (ValueError, lambda: q.qlinear_gated_forward(d, dh, w, w)),
            (ValueError, lambda: q.qlinear_gated_forward(d, x, w, small)),
            (ValueError, lambda: q.qlinear_gated_forward(d, x, w, dict(w, scales=None))),
            (ValueError, lambda: q.qlinear_gated_forward(d, x, w, w, act="relu")),
            (ValueError, lambda: q.qlinear_backward(d, x, w)),
            (ValueError, lambda: q.qlinear_backward(d, dh, small)),
            (ValueError, lambda: q.qlinear_gated_backward(d, dh, w, w, ok, (ok[0][:2], ok[1]))),
            (TypeError, lambda: q.qlinear_gated_backward(d, dh, w, w, ok, (ok[0].float(), ok[1])))):
        with pytest.raises(err):
            call()
