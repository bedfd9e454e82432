"""GPU tests of the MLP-block operators at the ends of their ranges, and over
long contractions under bounds that one lost step of 64 columns breaks.

Tolerances as in test_gpu_mlp.py, whose helpers are used here.
"""
import numpy as np
import pytest

import oracle
from oracle import mlp
from test_gpu_mlp import DT, TINY, U, dev, f64, packed, q, rel_limit, within  # noqa: F401  (q: the fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


# ---------------------------------------------------------------- small weights
# fp16 keeps weights down to 2^-14 = 6.1e-5 in full and then steps of 2^-24:
# rounding to the nearest costs at most 2^-25 each, 2^-25 / sqrt(3) in the rms,
# so weights of std 1e-4 lose 1.7e-4 of themselves that way, under a tenth of
# the 2e-3; the scales (down to 1e-6) may lose no more than their own rounding.
@pytest.mark.parametrize("std", [6e-4, 3e-4, 2e-4, 1e-4])
@pytest.mark.parametrize("meta", ["bf16", "f16"])
def test_backward_of_small_int8_weights(q, std, meta):
    rng = np.random.default_rng(int(std * 1e6))
    M, N, K = 40, 320, 256
    for gs in (32, 64, 128):
        print("small int8", std, meta, gs, flush=True)
        d = q.QDesc.affine(N, K, 8, gs, meta)
        (bg, wg), (bu, wu) = packed(q, d, rng, std), packed(q, d, rng, std)
        dy, dy64 = dev(rng.normal(size=(M, N)), "bf16")
        ref = dy64 @ wg
        assert oracle.rel_l2(f64(q.qlinear_backward(d, dy, bg, dx_dtype="f32")), ref) <= 2e-3
        ck = []
        for _ in range(2):
            c, s = mlp.checkpoint(rng.normal(size=(M, N)) * 2)
            ck.append((c, s, torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()))
        g, u = (mlp.restore(c[0], c[1]) for c in ck)
        o = q.qlinear_gated_backward(d, dy, bg, bu, ck[0][2:], ck[1][2:], dx_dtype="f32")
        dx, _, _ = mlp.gated_backward(dy64, g, u, wg, wu, "silu")
        assert oracle.rel_l2(f64(o.dx), dx) <= 2e-3


# ---------------------------------------------------------------- not finite
BAD = (float("nan"), float("inf"), float("-inf"))


def restored(q, ck):
    return f64(q.qpack_checkpoint_restore(ck, "f32"))


@pytest.mark.parametrize("K", [8, 64, 200, 1024, 65, 333])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_checkpoint_keeps_what_is_not_finite(q, K, dt):
    """A NaN or an infinity makes its group of 64 columns NaN, and no other."""
    rng = np.random.default_rng(K)
    M = 70
    x = torch.from_numpy(rng.normal(size=(M, K))).to(DT[dt])
    y, bad = x.clone(), np.zeros((M, K), bool)
    for m in range(0, M, 3):
        k = int(rng.integers(0, K))
        y[m, k] = BAD[(m // 3) % 3]
        bad[m, k // 64 * 64:k // 64 * 64 + 64] = True
    ck = q.qpack_checkpoint(y.cuda())
    clean, got = restored(q, q.qpack_checkpoint(x.cuda())), restored(q, ck)
    assert np.all(np.isnan(got[bad])) and np.array_equal(got[~bad], clean[~bad])
    assert not ck[0].cpu().numpy()[bad].any()


@pytest.mark.parametrize("K", [128, 100])
def test_every_nan_of_fp16_is_kept(q, K):
    """All 2046 NaN patterns, restored into each type."""
    bits = np.array([p for p in range(0x10000) if (p & 0x7C00) == 0x7C00 and p & 0x3FF], dtype=np.uint16)
    x = np.zeros((bits.size, K), dtype=np.uint16)
    x[np.arange(bits.size), np.arange(bits.size) % 64] = bits
    ck = q.qpack_checkpoint(torch.from_numpy(x.view(np.int16)).cuda().view(torch.float16))
    for od in ("f32", "bf16", "f16"):
        y = q.qpack_checkpoint_restore(ck, od)
        assert torch.isnan(y[:, :64]).all() and not y[:, 64:].any(), od


# stored as lines, as 4-column pieces and value by value; shares along K joined
@pytest.mark.parametrize("M,N,K", [(300, 208, 256), (300, 196, 256), (300, 201, 256), (20, 200, 2048)])
def test_gated_checkpoints_keep_what_is_not_finite(q, M, N, K):
    """A bias that is not finite: the outputs of its feature, and its group of
    64 in that layer's checkpoint; a row of x that is not: the whole row."""
    rng = np.random.default_rng(N)
    d = q.QDesc.affine(N, K, 4, 64, "bf16")
    (bg, _), (bu, _) = packed(q, d, rng), packed(q, d, rng)
    x = torch.from_numpy(rng.normal(size=(M, K))).bfloat16().cuda()
    c = torch.from_numpy(rng.normal(size=(2, N))).bfloat16()
    ref = q.qlinear_gated_forward(d, x, bg, bu, bias_gate=c[0].cuda(), bias_up=c[1].cuda(), save=True)
    for v in BAD:
        print("not finite", M, N, K, v, flush=True)
        b, xx = c.clone(), x.clone()
        b[0, 3], b[1, 77] = v, v
        xx[5, 9] = v
        o = q.qlinear_gated_forward(d, xx, bg, bu, bias_gate=b[0].cuda(), bias_up=b[1].cuda(), save=True)
        for ck, base, f in ((o.gate, ref.gate, 3), (o.up, ref.up, 77)):
            bad = np.zeros((M, N), bool)
            bad[5] = True
            bad[:, f // 64 * 64:f // 64 * 64 + 64] = True
            got = restored(q, ck)
            assert np.all(np.isnan(got[bad])) and np.array_equal(got[~bad], restored(q, base)[~bad])
        keep = np.ones((M, N), bool)
        keep[5] = False
        keep[:, [3, 77]] = False
        assert np.array_equal(f64(o.h)[keep], f64(ref.h)[keep])
        # into the gradients: the row, and nothing but the groups elsewhere
        g = q.qlinear_gated_backward(d, ref.h, bg, bu, o.gate, o.up)
        assert torch.isnan(g.dx).all()          # every row has such a group
        e = q.qlinear_gated_backward(d, ref.h, bg, bu, ref.gate, ref.up)
        far = np.ones((M, N), bool)
        far[5] = False
        far[:, :128] = False
        assert np.array_equal(f64(g.dgate)[far], f64(e.dgate)[far])


# ---------------------------------------------------------------- subnormal scales
@pytest.mark.parametrize("N,K", [(208, 256), (196, 256), (201, 256), (200, 2048)])
def test_gated_checkpoints_of_tiny_groups(q, N, K):
    """Rows of zeros leave g and u equal to the biases: groups whose scale is
    subnormal keep their codes, and their zeros."""
    rng = np.random.default_rng(N + 1)
    d = q.QDesc.affine(N, K, 4, 64, "bf16")
    (bg, _), (bu, _) = packed(q, d, rng), packed(q, d, rng)
    M = 20 if K > 256 else 150
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    for top in (1e-30, 3e-37, 1e-37, 3e-39, 1e-40):
        print("tiny", N, K, top, flush=True)
        c = rng.uniform(-1, 1, size=(2, N)) * top
        c[:, ::5] = 0
        b, b64 = dev(c, "bf16")
        o = q.qlinear_gated_forward(d, x, bg, bu, bias_gate=b[0].clone(), bias_up=b[1].clone(), save=True)
        for (codes, sc), v in ((o.gate, b64[:1]), (o.up, b64[1:])):
            rq, rs = mlp.checkpoint(v)
            assert np.array_equal(sc.cpu().numpy(), np.repeat(rs, M, 0))
            got = codes.cpu().numpy().astype(int)
            # a fp32 reciprocal: 127 steps at 3 * 2^-24, so a neighbour at a tie only
            assert np.all(np.abs(got - rq) <= 1) and not got[:, v[0] == 0].any()
            assert np.mean(got != rq) <= 0.02


# ---------------------------------------------------------------- the norm's range
@pytest.mark.parametrize("K", [256, 250, 4096, 40000])
def test_norm_products_past_fp32(q, K):
    """s * weight past fp32's range, or below its normal numbers, where the
    normed values are ordinary ones."""
    rng = np.random.default_rng(K)
    for sx, sw, eps in ((2e38, 1.0, 1e-5), (1e30, 1e20, 1e-5), (1e-25, 1e-15, 2.0 ** -126), (1e-28, 1e-12, 2.0 ** -126),
                        (1e30, 1e-30, 1e-5)):
        print("norm range", K, sx, sw, flush=True)
        x, x64 = dev(rng.uniform(-1, 1, size=(5, K)) * sx, "bf16")
        r, r64 = dev(rng.uniform(-0.2, 0.2, size=(5, K)) * sx, "bf16")
        w, w64 = dev(sw * (1 + rng.uniform(0, 3, size=K)), "bf16")
        for res in (None, r):
            s64 = x64 if res is None else f64(torch.from_numpy(x64 + r64).bfloat16())
            ref = mlp.norm(s64, w64, eps)
            into = {} if res is None else dict(residual=res, s_out=x.clone())
            o = q.qnorm_forward(into.get("s_out", x), w, eps=eps, **into)
            assert np.array_equal(f64(o.s), s64)
            within(o.y, ref, (U["bf16"] + 2.0 ** -21) * np.abs(ref) + TINY["bf16"], "y")
            p = q.qnorm_forward(x, w, residual=res, eps=eps, quantize=True)
            _, ys = mlp.row_codes(ref)
            within(p.ys, ys.astype(np.float64), 2.0 ** -23 * ys, "ys")
            step = f64(p.ys)[:, None]
            assert np.all(np.abs(ref - f64(p.yq) * step) <= (0.5 + 1e-9) * step)


@pytest.mark.parametrize("K", [256, 250, 4096])
@pytest.mark.parametrize("eps", [1e-5, 1e-20])
def test_norm_of_zeros(q, K, eps):
    """Rows of zeros, and rows under weights of zero."""
    x = torch.randn((6, K), device="cuda").bfloat16()
    x[2:4] = 0
    w = torch.ones(K, device="cuda").bfloat16()
    for wt, rows in ((w, slice(2, 4)), (0 * w, slice(0, 6))):
        o, p = q.qnorm_forward(x, wt, eps=eps), q.qnorm_forward(x, wt, eps=eps, quantize=True)
        assert not o.y[rows].any() and not p.yq[rows].any() and not p.ys[rows].any()
        assert torch.isfinite(o.y.float()).all()


@pytest.mark.parametrize("K", [256, 250, 4096])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_norm_keeps_what_is_not_finite(q, K, dt):
    """A row with a NaN or an infinity: NaN in its 16-bit row, NaN as the int8
    row's scale, and the other rows as they are."""
    rng = np.random.default_rng(K)
    x = torch.from_numpy(rng.normal(size=(7, K))).to(DT[dt])
    ref, refq = q.qnorm_forward(x.cuda()).y, q.qnorm_forward(x.cuda(), quantize=True)
    for m, v in ((1, float("nan")), (3, float("inf")), (5, float("-inf"))):
        x[m, K // 3] = v
    o, p = q.qnorm_forward(x.cuda()).y, q.qnorm_forward(x.cuda(), quantize=True)
    assert torch.isnan(o[[1, 3, 5], K // 3]).all() and torch.isnan(p.ys[[1, 3, 5]]).all()
    for a, b in ((o, ref), (p.yq, refq.yq), (p.ys, refq.ys)):
        assert torch.equal(a[::2], b[::2])


# ---------------------------------------------------------------- long contractions
def spread(D, w):
    """What a product's error stays under when its terms' roundings do not all
    point the same way.  Each term D w carries e with |e| <= 2^-11 |D w| from
    the weight and as much from D, 2^-11 / sqrt(3) each in the rms at worst;
    their signs go with D's, which are random here, so the sum's deviation is
    at most 2^-11 sqrt(2/3 sum D^2 w^2), of which ten are allowed: 8.2 of
    2^-11 sqrt(...), taken as 10.  Weights under fp16's normal range: 2^-25
    each.  fp32 sums: 2^-24 of a partial sum, sqrt(n) of them, under 2^-16 of
    the same root for n <= 65536."""
    return 10 * (2.0 ** -11 + 2.0 ** -16) * np.sqrt((D * D) @ (w * w)) + \
        10 * 2.0 ** -24 * np.sqrt(np.sum(D * D, axis=1, keepdims=True)) + 1e-30


def two_or_three(q, N, K):
    D = q.QDesc
    out = [D.affine(N, K, 4, 64, "bf16"), D.affine(N, K, 8, 32, "f16"), D.sym4(N, K)]
    return out + ([D.q4k(N, K), D.q6k(N, K)] if K % 256 == 0 else [])


@pytest.mark.parametrize("M,N,K,save", [
    (1, 20, 65536, False), (4, 20, 65536, True), (1, 37, 16384, True), (1, 37, 16384, False), (6, 35, 4096, True),
    (2, 37, 5120, True), (17, 33, 8192, False), (130, 40, 8192, True), (300, 24, 16384, False), (5, 70, 8224, True)])
def test_gated_forward_long(q, M, N, K, save):
    rng = np.random.default_rng(M + K)
    formats = two_or_three(q, N, K) if K % 64 == 0 else [q.QDesc.affine(N, K, 4, 32, "bf16")]
    for i, d in enumerate(formats):
        dt = ("bf16", "f16")[i % 2]
        print("gated long", M, N, K, d.fmt, d.bits, dt, save, flush=True)
        (bg, wg), (bu, wu) = packed(q, d, rng, 0.02), packed(q, d, rng, 0.02)
        x, x64 = dev(rng.normal(size=(M, K)), dt)
        o = q.qlinear_gated_forward(d, x, bg, bu, h_dtype="f32", save=save)
        g, u, h = mlp.gated(x64, wg, wu, 0.0, 0.0, "silu")
        dg, du = spread(x64, wg.T), spread(x64, wu.T)
        tol = 1.13 * dg * (np.abs(u) + du) + np.abs(mlp.act(g, "silu")[0]) * du + 2.0 ** -17 * np.abs(h) + 1e-30
        within(o.h, h, tol, "h")
        # the bound is one: without any step of 64 columns the result breaks it
        for t in (0, K // 128, (K - 1) // 64):
            keep = np.ones(K)
            keep[64 * t:64 * t + 64] = 0
            lost = mlp.gated(x64 * keep, wg, wu, 0.0, 0.0, "silu")[2]
            assert np.any(np.abs(lost - h) > 2 * tol)
        if save:
            for (codes, sc), v, e in ((o.gate, g, dg), (o.up, u, du)):
                step = np.repeat(f64(sc), 64, axis=1)[:, :N]
                got = mlp.restore(codes.cpu().numpy(), sc.cpu().numpy())
                assert np.all(np.abs(got - v) <= (0.5 + 1e-4) * step + e)


# rows of 1 to 8 chunks per thread in the staging kernel, and past its longest
BACK = [(5, 1800, 256), (33, 4000, 320), (9, 6000, 512), (130, 14336, 256), (7, 20000, 256), (6, 33000, 256),
        (3, 3001, 320)]


@pytest.mark.parametrize("M,N,K", BACK)
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_backward_long(q, M, N, K, kind):
    rng = np.random.default_rng(M + N)
    for i, d in enumerate(two_or_three(q, N, K)[(0 if kind == "silu" else 1)::2]):
        dt = ("bf16", "f16")[i % 2]
        print("backward long", M, N, K, d.fmt, d.bits, dt, kind, flush=True)
        (bg, wg), (bu, wu) = packed(q, d, rng), packed(q, d, rng)
        dh, dh64 = dev(rng.normal(size=(M, N)) * 1e-2, dt)
        ck = []
        for _ in range(2):
            c, s = mlp.checkpoint(rng.normal(size=(M, N)) * 2)
            ck.append((c, s, torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()))
        g, u = (mlp.restore(c[0], c[1]) for c in ck)
        o = q.qlinear_gated_backward(d, dh, bg, bu, ck[0][2:], ck[1][2:], act=kind, dx_dtype="f32")
        dx, rg, ru = mlp.gated_backward(dh64, g, u, wg, wu, kind)
        e = 2.0 ** -17       # fp32 chains of fewer than 16 operations around one exponential
        tg, tu = e * np.abs(dh64 * u) * (1 + np.abs(g)), e * np.abs(dh64) * (1 + np.abs(g))
        within(o.dgate, rg, U[dt] * np.abs(rg) + tg + TINY[dt], "dgate")
        within(o.dup, ru, U[dt] * np.abs(ru) + tu + TINY[dt], "dup")
        # their part of dx: 2^-17 of terms with dh's random signs, ten deviations
        chains = 10 * np.sqrt((tg * tg) @ (wg * wg) + (tu * tu) @ (wu * wu))
        both, w2 = np.concatenate([rg, ru], axis=1), np.concatenate([wg, wu])
        within(o.dx, dx, spread(both, w2) + chains + 2.0 ** -24 * np.abs(dx), "dx")
        assert oracle.rel_l2(f64(o.dx), dx) <= 2e-3
        one = q.qlinear_backward(d, dh, bg, dx_dtype="f32")
        ref = dh64 @ wg
        within(one, ref, spread(dh64, wg) + 2.0 ** -24 * np.abs(ref), "dx of one layer")
        assert oracle.rel_l2(f64(one), ref) <= rel_limit(ref, "f32", 2e-3)
        # the bound is one: without any step of 64 rows of W the result breaks it
        for t in (0, N // 128, (N - 1) // 64):
            lost = dh64[:, 64 * t:64 * t + 64] @ wg[64 * t:64 * t + 64]
            assert np.any(np.abs(lost) > 2 * spread(dh64, wg))
