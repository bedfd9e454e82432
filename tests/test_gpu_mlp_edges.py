"""GPU tests of the MLP-block operators at the ends of their ranges.

Tolerances as in test_gpu_mlp.py, whose helpers are used here.
"""
import numpy as np
import pytest

import oracle
from oracle import mlp
from test_gpu_mlp import DT, TINY, U, dev, f64, packed, q, within  # noqa: F401  (q: the fixture)

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
