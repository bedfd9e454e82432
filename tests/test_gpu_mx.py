"""GPU parity of MXFP4 weights and activations with their NumPy statement.

Tolerances.  Codes and scales are bit-exact.  Products of two MXFP4 values, or
of one and a 16-bit one, are exact in fp32, so only the sums round: an
addition by 2^-24 of its result (2^-23 where a matrix instruction truncates),
each at most the sum of the terms' magnitudes.  The few-row kernel adds 32
terms inside a chunk, the row's chunks, and at most 24 partial sums of lanes
and waves; the scaled matrix cores 64 inside an instruction and one
instruction after the other.  The staged forms round activations (and, out of
fp16's range, weights) to fp16: product_tolerance.
"""
import numpy as np
import pytest

import oracle
from oracle import mlp, mx
from test_gpu_mlp import DT, TINY, U, dev, f64, product_tolerance, rel_limit, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def q():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from bit_weight_only_qlinear_amd import qlinear
    return qlinear


def mx_rows(rng, N, K, scale=0.05, spread=0):
    """(codes, scales) of random rows and their fp64 values; spread: the blocks' sizes differ by up to 2^spread."""
    v = rng.normal(size=(N, K)) * scale
    if spread:
        v *= np.repeat(np.exp2(rng.integers(-spread, spread + 1, size=(N, K // 32))), 32, axis=1)
    c, s = mx.quantize(v)
    return c, s, mx.dequantize(c, s)


def on_gpu(c, s):
    return dict(qweight=torch.from_numpy(mx.pack(c).view(np.int32)).cuda(), scales=torch.from_numpy(s).cuda())


def layer(q, rng, N, K, **kw):
    c, s, w64 = mx_rows(rng, N, K, **kw)
    return q.QDesc.mxfp4(N, K), on_gpu(c, s), w64


def few_tol(x64, w64):
    K = w64.shape[1]
    return (32 + K // 32 + 24) * 2.0 ** -23 * (np.abs(x64) @ np.abs(w64).T)


def mxmx_tol(x64, w64):
    K = w64.shape[1]
    return (64 + K // 64 + 24) * 2.0 ** -23 * (np.abs(x64) @ np.abs(w64).T)


# ---------------------------------------------------------------- rows
def bits_of(t):
    return t.cpu().numpy().view(np.uint8 if t.element_size() == 1 else np.uint32)


@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (1, 4096), (7, 96), (33, 544), (130, 14336)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_quantize(q, M, K, dt):
    print("quantize", M, K, dt, flush=True)
    rng = np.random.default_rng(M * K)
    v = rng.normal(size=(M, K)) * 10.0 ** rng.uniform(-6, 4, size=(M, 1))
    x, x64 = dev(v, dt)
    c, s = mx.quantize(x64)
    gc, gs = q.quantize_activations_mx(x)
    assert np.array_equal(bits_of(gs), s) and np.array_equal(bits_of(gc), mx.pack(c))
    d = q.QDesc.mxfp4(M, K)
    if dt == "f32":
        w = q.qpack_quantize(d, x)
        assert torch.equal(w["qweight"], gc.view(-1)) and torch.equal(w["scales"], gs.view(-1))
        assert np.array_equal(q.qpack_unpack_codes(d, w).cpu().numpy(), c)
        p = q.qpack_pack_codes(d, torch.from_numpy(c).cuda())
        assert torch.equal(p["qweight"], gc.view(-1))
    for od in ("f32", "bf16", "f16"):
        got = q.qpack_dequantize(d, dict(qweight=gc, scales=gs), od)
        ref = torch.from_numpy(mx.dequantize(c, s)).float().to(DT[od])
        assert torch.equal(got.cpu(), ref), od


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_quantize_every_value(q, dt):
    """Every 16-bit pattern, in blocks whose largest value is at most 16 times
    as large, as large, or the pattern's own block of neighbours."""
    b = np.arange(1 << 16, dtype=np.uint16)
    v = torch.from_numpy(b.view(np.int16)).view(DT[dt])
    rows = [v.reshape(-1, 32)]
    for k in (1, 2, 4, 16):       # pairs (value, k times it) with zeros
        r = torch.zeros((1 << 16, 32), dtype=DT[dt])
        r[:, 3], r[:, 30] = v, -(v.float() * k).to(DT[dt])
        rows.append(r)
    x = torch.cat(rows)
    c, s = mx.quantize(f64(x))
    gc, gs = q.quantize_activations_mx(x.cuda())
    assert np.array_equal(bits_of(gs), s)
    assert np.array_equal(bits_of(gc), mx.pack(c))


def test_quantize_fp32_edges(q):
    """Powers of two and their neighbours over the whole range, ties, subnormals, infinities and NaN."""
    rng = np.random.default_rng(2)
    e = np.exp2(np.arange(-149, 128, dtype=np.float64))
    v = np.concatenate([e, e * (1 - 2.0 ** -24), e * 1.5, e * 1.75, e * 1.875, [0.0, -0.0, np.inf, -np.inf, np.nan]])
    with np.errstate(over="ignore"):
        v = v.astype(np.float32)
    x = np.zeros((len(v), 64), np.float32)
    x[:, 7] = v
    x[:, 8] = -v / 3
    x[:, 9] = v / 4
    x[:, 10] = v * np.float32(0.3125)
    x[:, 32:] = rng.normal(size=(len(v), 32)) * np.where(np.isfinite(v), v, 1)[:, None] / 4
    c, s = mx.quantize(x.astype(np.float64))
    gc, gs = q.quantize_activations_mx(torch.from_numpy(x).cuda())
    assert np.array_equal(bits_of(gs), s)
    assert np.array_equal(bits_of(gc), mx.pack(c))
    d = q.QDesc.mxfp4(len(v), 64)
    back = q.qpack_dequantize(d, dict(qweight=gc, scales=gs), "f32").cpu().numpy()
    assert np.array_equal(back, mx.dequantize(c, s).astype(np.float32), equal_nan=True)


def test_concat(q):
    rng = np.random.default_rng(3)
    ds, ws, vs = zip(*[layer(q, rng, n, 96) for n in (5, 64, 1)])
    d, w = q.concat_n(ds, ws)
    assert d.N == 70
    assert np.array_equal(f64(q.qpack_dequantize(d, w)), np.concatenate(vs))


# ---------------------------------------------------------------- 16-bit activations
FEW = [(1, 1, 32), (1, 17, 64), (2, 48, 96), (4, 33, 512), (5, 100, 544), (8, 64, 1024), (9, 16, 1056),
       (16, 257, 2048), (1, 130, 4096), (3, 70, 8224), (13, 40, 14336), (1, 33, 65536), (17, 50, 96), (40, 31, 160)]


@pytest.mark.parametrize("M,N,K", FEW)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_few_rows(q, M, N, K, dt):
    rng = np.random.default_rng(M + N + K)
    d, w, w64 = layer(q, rng, N, K, spread=3)
    x, x64 = dev(rng.normal(size=(M, K)), dt)
    b, b64 = dev(rng.normal(size=N), dt)
    tol = few_tol(x64, w64)
    for yd, bias in (("f32", None), (dt, b), ("f16" if dt == "bf16" else "bf16", None)):
        print("few", M, N, K, dt, yd, flush=True)
        y = q.qlinear_forward(d, x, w, bias=bias, y_dtype=yd, kernel=q.QP_KERNEL_GEMV)
        ref = x64 @ w64.T + (0 if bias is None else b64)
        within(y, ref, tol * (1 + U[yd]) + (U[yd] + 2.0 ** -23) * np.abs(ref) + TINY[yd], yd)
        if M <= 16 or K % 64:
            assert torch.equal(y, q.qlinear_forward(d, x, w, bias=bias, y_dtype=yd))
    # both selectors
    assert torch.equal(q.qlinear_forward(d, x, w, y_dtype="f32", kernel=q.QP_KERNEL_GEMV_MFMA),
                       q.qlinear_forward(d, x, w, y_dtype="f32", kernel=q.QP_KERNEL_GEMV))


@pytest.mark.parametrize("M,N,K", [(17, 64, 64), (33, 200, 320), (130, 257, 512), (300, 14, 1024), (64, 70, 16384),
                                   (260, 300, 4096), (300, 5000, 1536)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gemm(q, M, N, K, dt):
    rng = np.random.default_rng(M * N)
    d, w, w64 = layer(q, rng, N, K, spread=2)
    v = rng.normal(size=(M, K))
    v[3] = 0
    if dt == "bf16":
        v[5] *= 1e20
    x, x64 = dev(v, dt)
    b, b64 = dev(rng.normal(size=N), dt)
    tol = product_tolerance(x64, w64.T)
    for yd, bias, ws in (("f32", None, "auto"), (dt, b, "auto"), ("f32", None, None)):
        print("gemm", M, N, K, dt, yd, ws, q.workspace_bytes(d, M), flush=True)
        if yd == "f16":
            pass
        y = q.qlinear_forward(d, x, w, bias=bias, y_dtype=yd, workspace=ws)
        ref = x64 @ w64.T + (0 if bias is None else b64)
        within(y, ref, tol * (1 + U[yd]) + (U[yd] + 2.0 ** -23) * np.abs(ref) + TINY[yd], yd)


@pytest.mark.parametrize("M,N,K", [(17, 64, 64), (33, 200, 320), (130, 257, 512), (300, 14, 1024), (64, 70, 16384),
                                   (260, 300, 4096)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gemm_by_name(q, M, N, K, dt):
    rng = np.random.default_rng(M * N + 1)
    d, w, w64 = layer(q, rng, N, K, spread=2)
    v = rng.normal(size=(M, K))
    v[3] = 0
    if dt == "bf16":
        v[5] *= 1e20
    x, x64 = dev(v, dt)
    tol = product_tolerance(x64, w64.T)
    ref = x64 @ w64.T
    for yd in ("f32", dt):
        y = q.qlinear_forward(d, x, w, y_dtype=yd, kernel=q.QP_KERNEL_GEMM)
        within(y, ref, tol * (1 + U[yd]) + (U[yd] + 2.0 ** -23) * np.abs(ref) + TINY[yd], yd)


@pytest.mark.parametrize("M,N,K", [(17, 300, 512), (70, 1000, 1088), (500, 33, 64), (257, 8200, 128), (9, 8300, 192),
                                   (33, 8250, 320), (16, 20, 94144), (13, 20, 98304), (40, 24, 30784), (64, 70, 14336),
                                   (9, 1, 64), (64, 16, 4096), (13, 40, 114656), (3, 40, 114656), (1000, 4096, 256), (100, 9000, 608)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_few_rows_take_many(q, M, N, K, dt):
    """AUTO up to M N = 2^22: exact codes, in tiles of 16 to 64 rows."""
    rng = np.random.default_rng(M + N)
    d, w, w64 = layer(q, rng, N, K, spread=3)
    x, x64 = dev(rng.normal(size=(M, K)), dt)
    assert q.workspace_bytes(d, M) == 0
    y = q.qlinear_forward(d, x, w, y_dtype="f32")
    ref = x64 @ w64.T
    within(y, ref, few_tol(x64, w64) + 2.0 ** -23 * np.abs(ref) + TINY["f32"], "f32")
    assert torch.equal(y, q.qlinear_forward(d, x, w, y_dtype="f32", kernel=q.QP_KERNEL_GEMV))


def test_scales_over_the_range(q):
    """Blocks at both ends of the scale byte, in the exact kernels."""
    N, K = 16, 64
    c = np.tile(np.arange(16, dtype=np.uint8), (N, K // 16))
    s = np.full((N, 2), 127, np.uint8)
    s[:, 0] = [0, 1, 2, 3, 20, 60, 100, 126, 127, 128, 150, 200, 230, 250, 251, 252]
    w = on_gpu(c, s)
    x = np.zeros((3, K))
    x[0, 1], x[1, 15], x[2, 33] = 1.0, 0.5, 2.0
    t, x64 = dev(x, "bf16")
    ref = x64 @ mx.dequantize(c, s).T
    y = f64(q.qlinear_forward(q.QDesc.mxfp4(N, K), t, w, y_dtype="f32"))
    assert np.array_equal(y, ref)
    xc, xs = mx.quantize(x64)
    y = f64(q.qlinear_forward_mx(q.QDesc.mxfp4(N, K), *[on_gpu(xc, xs)[k] for k in ("qweight", "scales")], w,
                                 y_dtype="f32"))
    assert np.array_equal(y, ref)


def test_nan_blocks_stay_in_their_rows(q):
    """A weight block with scale 255 makes its output column NaN, an activation
    row with one its output row; nothing else."""
    rng = np.random.default_rng(7)
    for M, N, K in ((3, 40, 160), (20, 300, 256), (70, 300, 256), (70, 40, 96)):
        print("nan", M, N, K, flush=True)
        c, s, w64 = mx_rows(rng, N, K)
        s[7, K // 32 - 1] = 255
        w = on_gpu(c, s)
        d = q.QDesc.mxfp4(N, K)
        x, _ = dev(rng.normal(size=(M, K)), "bf16")
        outs = [q.qlinear_forward(d, x, w), q.qlinear_gated_forward(d, x, w, w).h,
                q.qlinear_gated_forward(d, x, w, w, save=True).h]
        xq, xs = q.quantize_activations_mx(x)
        outs.append(q.qlinear_forward_mx(d, xq, xs, w))
        for i, y in enumerate(outs):
            bad = torch.isnan(y).cpu().numpy()
            assert bad[:, 7].all() and bad.sum() == M, i
        xs[1, 0] = 255
        bad = torch.isnan(q.qlinear_forward_mx(d, xq, xs, w)).cpu().numpy()
        assert bad[:, 7].all() and bad[1].all() and bad.sum() == M + N - 1


# ---------------------------------------------------------------- both operands in 4 bits
MXMX = FEW + [(17, 64, 128), (64, 300, 256), (65, 257, 384), (128, 130, 512), (129, 96, 640), (300, 513, 1152),
              (600, 1000, 256), (33, 50, 8192), (257, 7, 2048)]


@pytest.mark.parametrize("M,N,K", MXMX)
def test_mx_times_mx(q, M, N, K):
    rng = np.random.default_rng(M + 3 * N + K)
    d, w, w64 = layer(q, rng, N, K, spread=4)
    xc, xs, x64 = mx_rows(rng, M, K, scale=1.0, spread=4)
    x = on_gpu(xc, xs)
    b = rng.normal(size=N).astype(np.float32)
    tol = mxmx_tol(x64, w64)
    for yd, bias in (("f32", None), ("bf16", torch.from_numpy(b).cuda()), ("f16", None)):
        print("mxmx", M, N, K, yd, flush=True)
        y = q.qlinear_forward_mx(d, x["qweight"], x["scales"], w, bias=bias, y_dtype=yd)
        ref = x64 @ w64.T + (0 if bias is None else b)
        within(y, ref, tol * (1 + U[yd]) + (U[yd] + 2.0 ** -23) * np.abs(ref) + TINY[yd], yd)


def test_mx_times_mx_is_exact_on_small_numbers(q):
    """Codes of 0.5 .. 6 with scales of 2^-2 .. 2^2: every sum is a multiple of
    2^-6 below 2^17, exact in fp32 in any order, so each lane's place is checked."""
    rng = np.random.default_rng(8)
    for M, N, K in ((16, 64, 1024), (20, 300, 256), (64, 256, 512), (130, 512, 384), (256, 256, 1024)):
        print("exact", M, N, K, flush=True)
        w, x = (rng.integers(0, 16, size=(r, K)).astype(np.uint8) for r in (N, M))
        ws, xs = (rng.integers(125, 130, size=(r, K // 32)).astype(np.uint8) for r in (N, M))
        t, p = on_gpu(w, ws), on_gpu(x, xs)
        y = q.qlinear_forward_mx(q.QDesc.mxfp4(N, K), p["qweight"], p["scales"], t, y_dtype="f32")
        assert np.array_equal(f64(y), mx.dequantize(x, xs) @ mx.dequantize(w, ws).T)


# Beyond 64 rows and 32 tiles of 64, 128 or 256 x 256 outputs, or where the scales of
# a tile of rows do not fit LDS: the tiled kernel.  K % 128 != 0 never is.
TILED = [(40, 300, 65536), (100, 8450, 256), (128, 8449, 128), (130, 8500, 384), (600, 4500, 640), (257, 8200, 512)]
UNTILED = [(130, 70, 96), (200, 33, 32), (70, 8500, 160), (5, 30, 95200), (20, 18, 63456), (40, 17, 31200),
           (5, 30, 95232), (20, 18, 63488), (40, 17, 31232)]


@pytest.mark.parametrize("M,N,K", TILED + UNTILED)
def test_mx_times_mx_by_size(q, M, N, K):
    rng = np.random.default_rng(M + 5 * N + K)
    d, w, w64 = layer(q, rng, N, K, spread=4)
    xc, xs, x64 = mx_rows(rng, M, K, scale=1.0, spread=4)
    x = on_gpu(xc, xs)
    b = rng.normal(size=N).astype(np.float32)
    tol, product = mxmx_tol(x64, w64), x64 @ w64.T
    for yd, bias in (("f32", torch.from_numpy(b).cuda()), ("bf16", None)):
        print("mxmx", M, N, K, yd, flush=True)
        y = q.qlinear_forward_mx(d, x["qweight"], x["scales"], w, bias=bias, y_dtype=yd)
        ref = product + (0 if bias is None else b)
        within(y, ref, tol * (1 + U[yd]) + (U[yd] + 2.0 ** -23) * np.abs(ref) + TINY[yd], yd)


def test_mx_times_mx_is_exact_at_every_size(q):
    """Small numbers as above, where every output tells its place."""
    rng = np.random.default_rng(18)
    for M, N, K in ((1, 70, 544), (33, 90, 96), (64, 8300, 512), (65, 100, 160), (100, 8450, 256), (130, 8500, 128),
                    (600, 4500, 640), (48, 33, 2080)):
        print("exact", M, N, K, flush=True)
        w, x = (rng.integers(0, 16, size=(r, K)).astype(np.uint8) for r in (N, M))
        ws, xs = (rng.integers(125, 130, size=(r, K // 32)).astype(np.uint8) for r in (N, M))
        t, p = on_gpu(w, ws), on_gpu(x, xs)
        y = q.qlinear_forward_mx(q.QDesc.mxfp4(N, K), p["qweight"], p["scales"], t, y_dtype="f32")
        assert np.array_equal(f64(y), mx.dequantize(x, xs) @ mx.dequantize(w, ws).T)


def test_nan_blocks_of_tiles_stay_in_their_rows(q):
    rng = np.random.default_rng(19)
    for M, N, K in ((130, 8500, 256), (1, 70, 96), (64, 33, 1056)):
        print("nan", M, N, K, flush=True)
        c, s, _ = mx_rows(rng, N, K)
        s[7, K // 32 - 1] = 255
        xc, xs, _ = mx_rows(rng, M, K)
        xs[M - 1, 0] = 255
        x = on_gpu(xc, xs)
        y = q.qlinear_forward_mx(q.QDesc.mxfp4(N, K), x["qweight"], x["scales"], on_gpu(c, s))
        bad = torch.isnan(y).cpu().numpy()
        assert bad[:, 7].all() and bad[M - 1].all() and bad.sum() == M + N - 1


# ---------------------------------------------------------------- gated pair and gradients
@pytest.mark.parametrize("M,N,K,save", [(1, 48, 512, False), (3, 100, 96, False), (8, 33, 4096, False),
                                        (16, 257, 544, False), (5, 70, 96, True), (17, 130, 512, False),
                                        (40, 33, 160, True), (300, 200, 512, True), (700, 5000, 256, False)])
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_gated(q, M, N, K, save, kind):
    rng = np.random.default_rng(M + N)
    dt = "bf16" if kind == "silu" else "f16"
    print("gated", M, N, K, save, kind, flush=True)
    (d, bg, wg), (_, bu, wu) = layer(q, rng, N, K), layer(q, rng, N, K)
    x, x64 = dev(rng.normal(size=(M, K)), dt)
    c1, c164 = dev(rng.normal(size=N) * 0.3, dt)
    c2, c264 = dev(rng.normal(size=N) * 0.3, dt)
    for hd in (dt, "f32"):
        o = q.qlinear_gated_forward(d, x, bg, bu, act=kind, bias_gate=c1, bias_up=c2, h_dtype=hd, save=save)
        g, u, h = mlp.gated(x64, wg, wu, c164, c264, kind)
        e = [product_tolerance(x64, v.T) if save or M > 16 else few_tol(x64, v) for v in (wg, wu)]
        dg, du = e[0] + 2.0 ** -22 * np.abs(g), e[1] + 2.0 ** -22 * np.abs(u)
        tol = 1.13 * dg * (np.abs(u) + du) + np.abs(mlp.act(g, kind)[0]) * du + \
            (U[hd] + 2.0 ** -17) * np.abs(h) + TINY[hd]
        within(o.h, h, tol, "h")
        if save:
            for (codes, sc), v, t in ((o.gate, g, dg), (o.up, u, du)):
                got = mlp.restore(codes.cpu().numpy(), sc.cpu().numpy())
                step = np.repeat(f64(sc), 64, axis=1)[:, :N]
                assert np.all(np.abs(got - v) <= (0.5 + 1e-4) * step + t)


@pytest.mark.parametrize("M,N,K", [(13, 20, 98304), (9, 18, 114656), (16, 20, 65568), (5, 17, 114656),
                                   (1, 17, 114656), (9, 18, 114688)])
def test_gated_long_rows(q, M, N, K):
    """Scales that leave no room for a step of 16 rows in LDS: tiles of eight."""
    rng = np.random.default_rng(M + N)
    (d, bg, wg), (_, bu, wu) = layer(q, rng, N, K), layer(q, rng, N, K)
    x, x64 = dev(rng.normal(size=(M, K)) * 0.05, "bf16")
    print("gated", M, N, K, flush=True)
    o = q.qlinear_gated_forward(d, x, bg, bu, act="silu", h_dtype="f32")
    none = np.zeros(N)
    g, u, h = mlp.gated(x64, wg, wu, none, none, "silu")
    dg, du = few_tol(x64, wg) + 2.0 ** -22 * np.abs(g), few_tol(x64, wu) + 2.0 ** -22 * np.abs(u)
    tol = 1.13 * dg * (np.abs(u) + du) + np.abs(mlp.act(g, "silu")[0]) * du + (U["f32"] + 2.0 ** -17) * np.abs(h) + TINY["f32"]
    within(o.h, h, tol, "h")


@pytest.mark.parametrize("M,N,K", [(1, 48, 256), (3, 100, 512), (17, 1, 96), (64, 63, 320), (130, 257, 512),
                                   (300, 192, 96), (5, 1000, 160), (260, 640, 320)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_backward(q, M, N, K, dt):
    rng = np.random.default_rng(N + K)
    (d, bg, wg), (_, bu, wu) = layer(q, rng, N, K), layer(q, rng, N, K)
    dy, dy64 = dev(rng.normal(size=(M, N)) * 1e-2, dt)
    for xd in (dt, "f32"):
        print("backward", M, N, K, dt, xd, flush=True)
        got = q.qlinear_backward(d, dy, bg, dx_dtype=xd)
        ref = dy64 @ wg
        within(got, ref, product_tolerance(dy64, wg) * (1 + U[xd]) + U[xd] * np.abs(ref) + TINY[xd], "dx")
        assert oracle.rel_l2(f64(got), ref) <= rel_limit(ref, xd, 2e-3)
    kind = "silu" if dt == "bf16" else "gelu_tanh"
    ck = [mlp.checkpoint(rng.normal(size=(M, N)) * 2) for _ in range(2)]
    g, u = (mlp.restore(*c) for c in ck)
    o = q.qlinear_gated_backward(d, dy, bg, bu, *[tuple(torch.from_numpy(a).cuda() for a in c) for c in ck],
                                 act=kind, dx_dtype="f32")
    dx, rg, ru = mlp.gated_backward(dy64, g, u, wg, wu, kind)
    e = 2.0 ** -17
    own = e * (np.abs(dy64 * u) * (1 + np.abs(g)) @ np.abs(wg) + np.abs(dy64) * (1 + np.abs(g)) @ np.abs(wu))
    tol = product_tolerance(np.concatenate([rg, ru], 1), np.concatenate([wg, wu])) + own
    within(o.dx, dx, tol + 2.0 ** -23 * np.abs(dx), "gated dx")


def test_gradient_against_differences(q):
    """The input gradient of sum(y * c) against differences of the exact forward."""
    rng = np.random.default_rng(10)
    M, N, K = 4, 48, 96
    d, w, w64 = layer(q, rng, N, K, scale=0.5)
    x = rng.integers(-8, 9, size=(M, K)).astype(np.float64)      # forwards are exact in fp32
    c = rng.integers(-4, 5, size=(M, N)).astype(np.float64)
    dx = f64(q.qlinear_backward(d, dev(c, "bf16")[0], w, dx_dtype="f32"))

    def loss(v):
        y = f64(q.qlinear_forward(d, dev(v, "bf16")[0], w, y_dtype="f32"))
        return (y * c).sum(axis=1)
    for k in (0, 31, 32, 95):
        hi, lo = x.copy(), x.copy()
        hi[:, k] += 1
        lo[:, k] -= 1
        assert np.allclose(dx[:, k], (loss(hi) - loss(lo)) / 2, rtol=1e-6, atol=1e-6)


# ---------------------------------------------------------------- together
def test_chain_captured_and_replayed(q):
    """A block with MXFP4 weights forward and backward, and its 4-bit-activation
    form, in one graph: every replay equals the eager result."""
    rng = np.random.default_rng(11)
    M, K, N = 24, 256, 320
    (d, bg, _), (_, bu, _), (dn, bn, _) = layer(q, rng, N, K), layer(q, rng, N, K), layer(q, rng, K, N)
    x, _ = dev(rng.normal(size=(M, K)), "bf16")
    dy, _ = dev(rng.normal(size=(M, K)) * 1e-2, "bf16")

    def step():
        n = q.qnorm_forward(x).y
        f = q.qlinear_gated_forward(d, n, bg, bu, save=True)
        y = q.qlinear_forward(dn, f.h, bn)
        gb = q.qlinear_gated_backward(d, q.qlinear_backward(dn, dy, bn), bg, bu, f.gate, f.up)
        a = q.quantize_activations_mx(n)
        z = q.qlinear_forward_mx(d, *a, bg)
        t = q.qlinear_forward_mx(d, a[0][:5], a[1][:5], bg)
        return [f.h, y, gb.dx, *a, z, t, q.qlinear_forward(d, n[:3], bg)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(4):
        for t in (x, dy):
            t.copy_(torch.from_numpy(rng.normal(size=t.shape)))
        eager = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, eager)):
            assert torch.equal(a, b), (k, i)


def test_two_streams(q):
    rng = np.random.default_rng(12)
    d, w, _ = layer(q, rng, 512, 1024)
    x = torch.randn((2, 200, 1024), device="cuda").bfloat16()

    def both(t):
        return q.qlinear_forward_mx(d, *q.quantize_activations_mx(t), w), q.qlinear_forward(d, t[:9], w)
    want = [both(x[i]) for i in range(2)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for i in range(2):
            with torch.cuda.stream(st[i]):
                got.append(both(x[i]))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, v in zip(got, want) for a, b in zip(g, v))


def test_outputs_stay_inside(q):
    """Bytes past the last row are left as they were."""
    rng = np.random.default_rng(13)
    K = 128
    for M, N in ((3, 21), (19, 70), (70, 300)):
        d, w, _ = layer(q, rng, N, K)
        x, _ = dev(rng.normal(size=(M, K)), "bf16")
        xq, xs = q.quantize_activations_mx(x)
        for dt in (torch.bfloat16, torch.float32):
            t = torch.full((M * N + 4096,), 77, dtype=dt, device="cuda")
            yd = "bf16" if dt == torch.bfloat16 else "f32"
            q.qlinear_forward_mx(d, xq, xs, w, y_dtype=yd, out=t[:M * N].view(M, N))
            assert torch.all(t[M * N:] == 77)
            t.fill_(77)
            q.qlinear_forward(d, x, w, y_dtype=yd, out=t[:M * N].view(M, N))
            assert torch.all(t[M * N:] == 77)
        t = torch.full((M * K // 8 + 64,), 7, dtype=torch.int32, device="cuda")
        s = torch.full((M * K // 32 + 64,), 7, dtype=torch.uint8, device="cuda")
        q._run(x.device, q.lib.qpack_quantize_activations_mx, x.data_ptr(), 1, M, K, t.data_ptr(), s.data_ptr())
        assert torch.all(t[M * K // 8:] == 7) and torch.all(s[M * K // 32:] == 7)
        assert torch.equal(t[:M * K // 8].view(M, -1), xq) and torch.equal(s[:M * K // 32].view(M, -1), xs)


def test_offsets_past_32_bits(q):
    """Buffers of more than 2^32 bytes: their last rows against the same rows alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    M, K = 140000, 16384
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    x[:] = torch.randn((1, K), device="cuda", generator=g)
    x[-300:] = torch.randn((300, K), device="cuda", generator=g)
    a, b = q.quantize_activations_mx(x), q.quantize_activations_mx(x[-300:].contiguous())
    assert torch.equal(a[0][-300:], b[0]) and torch.equal(a[1][-300:], b[1])
    v = q.qpack_dequantize(q.QDesc.mxfp4(M, K), dict(qweight=a[0], scales=a[1]), "bf16")
    w = q.qpack_dequantize(q.QDesc.mxfp4(300, K), dict(qweight=b[0], scales=b[1]), "bf16")
    assert torch.equal(v[-300:], w)
    del v, w, x
    # the rows as weights, more than 2^30 codes' bytes; and as activations
    d = q.QDesc.mxfp4(M, K)
    t = torch.randn((3, K), device="cuda", generator=g).bfloat16()
    W = dict(qweight=a[0], scales=a[1])
    y = q.qlinear_forward(d, t, W)
    z = q.qlinear_forward(q.QDesc.mxfp4(300, K), t, dict(qweight=b[0], scales=b[1]))
    assert torch.equal(y[:, -300:], z)
    s = q.QDesc.mxfp4(20000, K)
    few = dict(qweight=a[0][-20000:], scales=a[1][-20000:])
    y = q.qlinear_forward_mx(s, *a, few)                      # 2.8e9 outputs
    z = q.qlinear_forward_mx(s, *b, few)
    assert torch.equal(y[-300:], z)


@pytest.mark.parametrize("M,N", [(9, 21), (13, 70), (33, 35), (64, 18), (40, 130), (100, 8451)])
def test_outputs_stay_inside_by_size(q, M, N):
    rng = np.random.default_rng(M)
    K = 160 if N < 1000 else 128
    d, w, _ = layer(q, rng, N, K)
    x, _ = dev(rng.normal(size=(M, K)), "f16")
    xq, xs = q.quantize_activations_mx(x)
    for dt, yd in ((torch.float16, "f16"), (torch.float32, "f32")):
        t = torch.full((M * N + 4096,), 77, dtype=dt, device="cuda")
        for f in (lambda o: q.qlinear_forward_mx(d, xq, xs, w, y_dtype=yd, out=o),
                  lambda o: q.qlinear_forward(d, x, w, y_dtype=yd, kernel=q.QP_KERNEL_GEMV, out=o)):
            t.fill_(77)
            f(t[:M * N].view(M, N))
            assert torch.all(t[M * N:] == 77) and not torch.any(t[:M * N] == 77)


def test_weights_past_32_bits(q):
    """Codes of more than 2^32 bytes: the last rows against the same rows alone (small
    numbers, whose sums are exact in any order)."""
    N, K, n = 560000, 16384, 50
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    codes = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), dtype=torch.int32, device="cuda", generator=g)
    scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    w, last = dict(qweight=codes, scales=scales), dict(qweight=codes[-n:], scales=scales[-n:])
    d, e = q.QDesc.mxfp4(N, K), q.QDesc.mxfp4(n, K)
    for M in (1, 6, 9, 33, 70):
        print("weights", M, flush=True)
        x = torch.randint(-2, 3, (M, K), device="cuda", generator=g).bfloat16()
        y = q.qlinear_forward(d, x, w, y_dtype="f32", kernel=q.QP_KERNEL_GEMV)
        assert torch.equal(y[:, -n:], q.qlinear_forward(e, x, last, y_dtype="f32", kernel=q.QP_KERNEL_GEMV))
        a = torch.randint(-2 ** 31, 2 ** 31, (M, K // 8), dtype=torch.int32, device="cuda", generator=g)
        b = torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda")
        y = q.qlinear_forward_mx(d, a, b, w, y_dtype="f32")
        assert torch.equal(y[:, -n:], q.qlinear_forward_mx(e, a, b, last, y_dtype="f32"))


def test_binding_refuses_wrong_tensors(q):
    d = q.QDesc.mxfp4(32, 64)
    w = q.qpack_quantize(d, torch.zeros((32, 64), device="cuda"))
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    xq, xs = q.quantize_activations_mx(x)
    for err, call in (
            (TypeError, lambda: q.quantize_activations_mx(x.double())),
            (ValueError, lambda: q.quantize_activations_mx(x.t())),
            (q.QLinearError, lambda: q.quantize_activations_mx(x[:, :48].contiguous())),
            (q.QLinearError, lambda: q.quantize_activations_mx(x[:0])),
            (TypeError, lambda: q.qlinear_forward_mx(d, xq.float(), xs, w)),
            (ValueError, lambda: q.qlinear_forward_mx(d, xq, xs[:2], w)),
            (ValueError, lambda: q.qlinear_forward_mx(d, xq[:, :4], xs, w)),
            (ValueError, lambda: q.qlinear_forward_mx(d, xq, xs, dict(w, scales=None))),
            (TypeError, lambda: q.qlinear_forward_mx(d, xq, xs, w, bias=x[0, :32])),
            (ValueError, lambda: q.qlinear_forward_mx(d, xq, xs, w, out=torch.empty((4, 31), device="cuda").bfloat16())),
            (ValueError, lambda: q.qlinear_forward_mx(d, xq, xs, w, y_dtype="f64"))):
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("M", [9, 10, 11, 12, 13, 15])
@pytest.mark.parametrize("N,K", [(70, 512), (33, 32), (130, 544), (40, 2048)])
def test_gated_of_nine_rows_and_more(q, M, N, K):
    """One tile of 16 rows that are not all there, whole rows of x in LDS."""
    rng = np.random.default_rng(M + N)
    (d, bg, wg), (_, bu, wu) = layer(q, rng, N, K), layer(q, rng, N, K)
    x, x64 = dev(rng.normal(size=(M, K)), "bf16")
    print("gated", M, N, K, flush=True)
    o = q.qlinear_gated_forward(d, x, bg, bu, act="silu", h_dtype="f32")
    g, u, h = mlp.gated(x64, wg, wu, np.zeros(N), np.zeros(N), "silu")
    dg, du = few_tol(x64, wg) + 2.0 ** -22 * np.abs(g), few_tol(x64, wu) + 2.0 ** -22 * np.abs(u)
    tol = 1.13 * dg * (np.abs(u) + du) + np.abs(mlp.act(g, "silu")[0]) * du + 2.0 ** -16 * np.abs(h) + TINY["f32"]
    within(o.h, h, tol, "h")


# ---------------------------------------------------------------- the qGEMM, by name and where AUTO takes it
def mx_tolerance(D, w, top):
    """Largest error of D [M, n] (rounded once to fp16: 2^-11 of each value, 2^-39 of
    its row's maximum for the smallest) times w [n, K], whose columns' fp16 numbers
    are multiples of 2^-37 of 2^top, a column's largest scale (fp16's last bit, 2^-24,
    where that scale becomes 2^13): half of that; the sums n + 32 additions of 2^-23 in
    instructions that truncate."""
    a, v = np.abs(D), np.abs(w)
    n = w.shape[0]
    return (2.0 ** -11 + (n + 32) * 2.0 ** -23) * (a @ v) + 2.0 ** -38 * a.sum(axis=1, keepdims=True) * np.exp2(top) + \
        2.0 ** -39 * a.max(axis=1, keepdims=True) * v.sum(axis=0)


def scales_from(rng, N, C, low, high, wide):
    """Scale bytes [N, C] of rows whose largest lie in low .. high, and up to `wide` below."""
    top = rng.integers(low, high + 1, size=(N, 1))
    s = top - rng.integers(0, wide + 1, size=(N, C))
    s[:, rng.integers(0, C)] = top[:, 0]
    return np.clip(s, 0, 254).astype(np.uint8)


QGEMM = [(17, 64, 64), (300, 257, 512), (33, 130, 1088), (257, 301, 1024), (16, 20, 192), (520, 250, 128), (40, 33, 64),
         (290, 225, 192)]


@pytest.mark.parametrize("M,N,K", QGEMM)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_qgemm_in_both_tilings(q, M, N, K, dt):
    """With a workspace where the call has a use for one, and without; a block of
    scale 255 keeps to its output column."""
    rng = np.random.default_rng(M + N + K)
    c = rng.integers(0, 16, size=(N, K)).astype(np.uint8)
    s = scales_from(rng, N, K // 32, 112, 124, 6)
    w64 = mx.dequantize(c, s)
    d, w = q.QDesc.mxfp4(N, K), on_gpu(c, s)
    x, x64 = dev(rng.normal(size=(M, K)), dt)
    b, b64 = dev(rng.normal(size=N), dt)
    ref = x64 @ w64.T + b64
    tol = mx_tolerance(x64, w64.T, s.max(axis=1) - 127.0)
    for ws in (None, "auto"):
        for yd in ("f32", dt):
            print("qgemm", M, N, K, dt, ws, yd, q.workspace_bytes(d, M, kernel=q.QP_KERNEL_GEMM), flush=True)
            y = q.qlinear_forward(d, x, w, bias=b, y_dtype=yd, kernel=q.QP_KERNEL_GEMM, workspace=ws)
            within(y, ref, tol * (1 + U[yd]) + (U[yd] + 2.0 ** -23) * np.abs(ref) + TINY[yd], yd)
        s2 = s.copy()
        s2[N - 1, 0] = s2[3, K // 32 - 1] = 255
        y2 = q.qlinear_forward(d, x, on_gpu(c, s2), bias=b, y_dtype="f32", kernel=q.QP_KERNEL_GEMM, workspace=ws)
        bad = torch.isnan(y2).cpu().numpy()
        assert bad[:, [3, N - 1]].all() and bad.sum() == 2 * M
        keep = [n for n in range(N) if n not in (3, N - 1)]
        within(y2[:, keep], ref[:, keep], (tol + 2.0 ** -22 * np.abs(ref))[:, keep] + TINY["f32"], "others")


@pytest.mark.parametrize("M,N,K,staged", [(257, 32763, 128, False), (300, 14336, 512, True), (290, 14500, 320, True)])
def test_auto_takes_the_qgemm(q, M, N, K, staged):
    """M N past 2^22: AUTO is the qGEMM, with a workspace or not."""
    rng = np.random.default_rng(M + N)
    c = rng.integers(0, 16, size=(N, K)).astype(np.uint8)
    s = scales_from(rng, N, K // 32, 112, 124, 6)
    w64 = mx.dequantize(c, s)
    d, w = q.QDesc.mxfp4(N, K), on_gpu(c, s)
    x, x64 = dev(rng.normal(size=(M, K)), "bf16")
    need = q.workspace_bytes(d, M)
    print("auto", M, N, K, need, flush=True)
    assert need == q.workspace_bytes(d, M, kernel=q.QP_KERNEL_GEMM) and staged == (need > 0)
    ref = x64 @ w64.T
    tol = mx_tolerance(x64, w64.T, s.max(axis=1) - 127.0) + 2.0 ** -23 * np.abs(ref) + TINY["f32"]
    for ws in (None, "auto"):
        y = q.qlinear_forward(d, x, w, y_dtype="f32", workspace=ws)
        within(y, ref, tol, "y")
        assert torch.equal(y, q.qlinear_forward(d, x, w, y_dtype="f32", kernel=q.QP_KERNEL_GEMM, workspace=ws))


# scale bytes of a row's (a column's) largest block: fp16 alone holds weights of 104 .. 140
RANGES = [(0, 8), (40, 60), (100, 107), (138, 143), (200, 236), (0, 236)]


@pytest.mark.parametrize("low,high", RANGES)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_qgemm_takes_every_scale(q, low, high, dt):
    for M, N, K in ((40, 70, 512), (300, 300, 576)):
        rng = np.random.default_rng(M + low)
        c = rng.integers(0, 16, size=(N, K)).astype(np.uint8)
        s = scales_from(rng, N, K // 32, low, high, 12)
        c[5], s[6] = 0, 0          # a row of zeros, and one of the smallest scale
        w64 = mx.dequantize(c, s)
        d, w = q.QDesc.mxfp4(N, K), on_gpu(c, s)
        x, x64 = dev(rng.normal(size=(M, K)) / 16, dt)
        b, b64 = dev(rng.normal(size=N), dt)
        ref = x64 @ w64.T
        tol = mx_tolerance(x64, w64.T, s.max(axis=1) - 127.0) + 2.0 ** -22 * np.abs(ref) + TINY["f32"]
        for ws in (None, "auto"):
            print("scales", M, N, K, low, high, dt, ws, flush=True)
            y = q.qlinear_forward(d, x, w, y_dtype="f32", kernel=q.QP_KERNEL_GEMM, workspace=ws)
            within(y, ref, tol, "y")
            y = q.qlinear_forward(d, x, w, bias=b, y_dtype="f32", kernel=q.QP_KERNEL_GEMM, workspace=ws)
            within(y, ref + b64, tol + 2.0 ** -23 * np.abs(ref + b64), "with bias")
        # the kernels on exact codes
        within(q.qlinear_forward(d, x, w, y_dtype="f32", kernel=q.QP_KERNEL_GEMV), ref,
               few_tol(x64, w64) + 2.0 ** -22 * np.abs(ref) + TINY["f32"], "exact codes")


def test_qgemm_takes_the_largest_rows_and_weights(q):
    """bf16 rows of 1e30 against weights of 1e-25, and the other way round: finite results."""
    rng = np.random.default_rng(21)
    N, K = 70, 512
    c = rng.integers(0, 16, size=(N, K)).astype(np.uint8)
    for M, up, byte in ((40, 1e30, 40), (40, 1e-28, 210), (300, 1e30, 40)):
        s = scales_from(rng, N, K // 32, byte - 2, byte + 2, 3)
        w64 = mx.dequantize(c, s)
        x, x64 = dev(rng.normal(size=(M, K)) * up, "bf16")
        ref = x64 @ w64.T
        for ws in (None, "auto"):
            y = q.qlinear_forward(q.QDesc.mxfp4(N, K), x, on_gpu(c, s), y_dtype="f32", kernel=q.QP_KERNEL_GEMM,
                                  workspace=ws)
            within(y, ref, mx_tolerance(x64, w64.T, s.max(axis=1) - 127.0) + 2.0 ** -22 * np.abs(ref), "y")


GATED_RANGES = [(20, 40), (100, 107), (110, 150)]


@pytest.mark.parametrize("low,high", GATED_RANGES)
@pytest.mark.parametrize("M,N,K,save", [(40, 70, 512, True), (20, 33, 96, False), (300, 200, 608, False),
                                        (3, 130, 1024, True), (700, 5000, 64, False)])
def test_gated_takes_every_scale(q, M, N, K, save, low, high):
    """The gate's scales over the range, the up projection's the other way (products of
    the two stay finite)."""
    rng = np.random.default_rng(M + low)
    c1, c2 = (rng.integers(0, 16, size=(N, K)).astype(np.uint8) for _ in range(2))
    s1 = scales_from(rng, N, K // 32, low, high, 12)
    s2 = scales_from(rng, N, K // 32, 254 - high - 12, 254 - low - 12, 12)
    w1, w2 = mx.dequantize(c1, s1), mx.dequantize(c2, s2)
    d = q.QDesc.mxfp4(N, K)
    x, x64 = dev(rng.normal(size=(M, K)) / 16, "bf16")
    print("gated scales", M, N, K, save, low, high, flush=True)
    o = q.qlinear_gated_forward(d, x, on_gpu(c1, s1), on_gpu(c2, s2), act="silu", h_dtype="f32", save=save)
    none = np.zeros(N)
    with np.errstate(over="ignore"):
        g, u, h = mlp.gated(x64, w1, w2, none, none, "silu")
    dg = mx_tolerance(x64, w1.T, s1.max(axis=1) - 127.0) + 2.0 ** -22 * np.abs(g)
    du = mx_tolerance(x64, w2.T, s2.max(axis=1) - 127.0) + 2.0 ** -22 * np.abs(u)
    with np.errstate(over="ignore"):
        a = np.abs(mlp.act(g, "silu")[0])
    # the logistic's argument and exponential: 2^-17 where it is not next to 0; below -80 it is under 2^-115
    tol = 1.13 * dg * (np.abs(u) + du) + a * du + 2.0 ** -16 * np.abs(h) + TINY["f32"] + \
        np.where(g < -80, 2.0 ** -100 * np.abs(u), 0)
    within(o.h, h, tol, "h")
    if save:
        for (codes, sc), v, t in ((o.gate, g, dg), (o.up, u, du)):
            got = mlp.restore(codes.cpu().numpy(), sc.cpu().numpy())
            step = np.repeat(f64(sc), 64, axis=1)[:, :N]
            assert np.all(np.abs(got - v) <= (0.5 + 1e-4) * step + t)


@pytest.mark.parametrize("low,high", RANGES)
@pytest.mark.parametrize("M,N,K", [(3, 70, 96), (40, 300, 512), (300, 130, 800), (5, 2100, 256), (130, 64, 32), (4, 2101, 96),
                                   (3, 33, 40960), (2, 1, 64)])
def test_backward_takes_every_scale(q, M, N, K, low, high):
    """Columns (32 of them share a scale byte) of every size, and rows of every size."""
    rng = np.random.default_rng(N + low)
    c = rng.integers(0, 16, size=(N, K)).astype(np.uint8)
    dy, dy64 = dev(rng.normal(size=(M, N)) / 16, "bf16")
    d = q.QDesc.mxfp4(N, K)
    for s in (np.ascontiguousarray(scales_from(rng, K // 32, N, low, high, 12).T), scales_from(rng, N, K // 32, low, high, 12)):
        w64 = mx.dequantize(c, s)
        print("gradient scales", M, N, K, low, high, flush=True)
        ref = dy64 @ w64
        tol = mx_tolerance(dy64, w64, np.repeat(s.max(axis=0) - 127.0, 32))
        for xd in ("f32", "bf16"):
            got = q.qlinear_backward(d, dy, on_gpu(c, s), dx_dtype=xd)
            within(got, ref, tol * (1 + U[xd]) + (U[xd] + 2.0 ** -22) * np.abs(ref) + TINY[xd], "dx")


@pytest.mark.parametrize("low,high", [(20, 40), (110, 150)])
@pytest.mark.parametrize("M,N,K", [(3, 70, 96), (300, 130, 544)])
def test_gated_backward_takes_every_scale(q, M, N, K, low, high):
    rng = np.random.default_rng(N + low)
    cs = [rng.integers(0, 16, size=(N, K)).astype(np.uint8) for _ in range(2)]
    s1 = np.ascontiguousarray(scales_from(rng, K // 32, N, low, high, 12).T)
    s2 = np.clip(s1.astype(int) + rng.integers(-6, 7, size=s1.shape), 0, 254).astype(np.uint8)
    wg, wu = mx.dequantize(cs[0], s1), mx.dequantize(cs[1], s2)
    dh, dh64 = dev(rng.normal(size=(M, N)) * 1e-2, "bf16")
    ck = [mlp.checkpoint(rng.normal(size=(M, N)) * 2) for _ in range(2)]
    g, u = (mlp.restore(*k) for k in ck)
    print("gated gradient scales", M, N, K, low, high, flush=True)
    o = q.qlinear_gated_backward(q.QDesc.mxfp4(N, K), dh, on_gpu(cs[0], s1), on_gpu(cs[1], s2),
                                 *[tuple(torch.from_numpy(a).cuda() for a in k) for k in ck], act="silu", dx_dtype="f32")
    dx, rg, ru = mlp.gated_backward(dh64, g, u, wg, wu, "silu")
    own = 2.0 ** -17 * (np.abs(dh64 * u) * (1 + np.abs(g)) @ np.abs(wg) + np.abs(dh64) * (1 + np.abs(g)) @ np.abs(wu))
    top = np.repeat(np.maximum(s1, s2).max(axis=0) - 127.0, 32)
    tol = mx_tolerance(np.concatenate([rg, ru], 1), np.concatenate([wg, wu]), top) + own
    within(o.dx, dx, tol + 2.0 ** -22 * np.abs(dx) + TINY["f32"], "gated dx")


def test_nan_blocks_in_gradients(q):
    """A weight block of scale 255 makes its 32 columns of every gradient NaN, and no others."""
    rng = np.random.default_rng(23)
    for M, N, K in ((5, 200, 96), (300, 130, 800)):
        c = rng.integers(0, 16, size=(N, K)).astype(np.uint8)
        s = scales_from(rng, N, K // 32, 112, 124, 6)
        s[N - 1, 1] = 255
        dy, _ = dev(rng.normal(size=(M, N)), "bf16")
        bad = torch.isnan(q.qlinear_backward(q.QDesc.mxfp4(N, K), dy, on_gpu(c, s))).cpu().numpy()
        assert bad[:, 32:64].all() and bad.sum() == 32 * M
