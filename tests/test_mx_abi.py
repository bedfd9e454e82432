"""Argument checks of the MXFP4 and mixture-of-experts entry points: every
refusal happens on the host, before any launch (CPU; the addresses are never
read)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

FAKE, OUT, OTHER, WS = 1 << 30, 1 << 32, 1 << 34, 1 << 36


@pytest.fixture(scope="module")
def q():
    from bit_weight_only_qlinear_amd import qlinear
    return qlinear


def _err(q):
    return q.lib.qpack_last_error().decode()


def test_descriptor(q):
    d = q.QDesc.mxfp4(7, 96)
    s = q.qpack_sizes(d)
    assert s == dict(qweight=7 * 48, qweight_hi=0, scales=21, zeros=0, steps=0)
    big = q.QDesc.mxfp4(256, 4096)
    assert 8 * sum(q.qpack_sizes(big).values()) / (256 * 4096) == 4.25
    out = (ctypes.c_size_t * 5)()
    for kw, status, msg in ((dict(K=48), 2, "32"), (dict(bits=8), 3, "bits"), (dict(gs=64), 3, "group_size"),
                            (dict(sb=256), 3, "super_block"), (dict(N=0), 2, "positive")):
        a = dict(bits=4, gs=32, sb=0, N=8, K=64) | kw
        c = q._Desc(q.QP_FMT_MXFP4, a["bits"], a["gs"], a["sb"], 0, 0, a["N"], a["K"])
        assert q.lib.qpack_sizes(ctypes.byref(c), out) == status and msg in _err(q), (kw, _err(q))


def test_forward_selectors(q):
    """Which calls the few-row kernel and the qGEMM take."""
    w = q._Weights(FAKE, None, FAKE, None, None)
    n = ctypes.c_size_t(7)

    def ws(N, K, M, kernel):
        return q.lib.qlinear_workspace_bytes(ctypes.byref(q.QDesc.mxfp4(N, K).c()), 1, M, kernel, ctypes.byref(n))
    assert ws(14336, 4096, 16, q.QP_KERNEL_AUTO) == 0 and n.value == 0
    assert ws(14336, 4096, 2048, q.QP_KERNEL_AUTO) == 0 and n.value == 2048 * 4096 * 2 + 2048 * 4
    assert ws(14336, 4096, 2048, q.QP_KERNEL_GEMV) == 0 and n.value == 0
    assert ws(64, 96, 2048, q.QP_KERNEL_AUTO) == 0 and n.value == 0        # K % 64: few-row tiles
    assert ws(64, 96, 64, q.QP_KERNEL_GEMM) == q.QP_EUNSUPPORTED
    assert ws(64, 1 << 17, 64, q.QP_KERNEL_GEMM) == 0                       # exact weights: any K to 2^20
    assert ws(1 << 26, 96, 1 << 24, q.QP_KERNEL_AUTO) == q.QP_EUNSUPPORTED and "2^34" in _err(q)
    assert ws(64, 64, 0, q.QP_KERNEL_AUTO) == q.QP_ESHAPE
    d = q.QDesc.mxfp4(64, 64).c()
    assert q.lib.qlinear_forward(ctypes.byref(d), FAKE, 1, 1, ctypes.byref(q._Weights(FAKE, None, None, None, None)),
                                 None, OUT, 1, None) == q.QP_EINVAL and "scales" in _err(q)
    # entry points of other formats
    assert q.lib.qpack_quantize_hqq(ctypes.byref(d), FAKE, ctypes.byref(w), 20, 0.7, 10.0, 1.01,
                                    None) == q.QP_EUNSUPPORTED
    assert q.lib.qpack_encode_nested(ctypes.byref(d), FAKE, None, ctypes.byref(w), None, None) == q.QP_EUNSUPPORTED
    assert q.lib.qlinear_forward_a8w4(ctypes.byref(d), FAKE, FAKE, 1, ctypes.byref(w), None, OUT, 1,
                                      None) == q.QP_EUNSUPPORTED


def test_quantize_activations_refusals(q):
    f = q.lib.qpack_quantize_activations_mx
    for a, status, msg in (
            ((FAKE, 3, 2, 64, OUT, OTHER), 1, "x_dtype"), ((FAKE, 1, 0, 64, OUT, OTHER), 2, "positive"),
            ((FAKE, 1, 2, 0, OUT, OTHER), 2, "positive"), ((FAKE, 1, 2, 48, OUT, OTHER), 2, "32"),
            ((FAKE, 1, 2, (1 << 24) + 32, OUT, OTHER), 3, "2^24"), ((None, 1, 2, 64, OUT, OTHER), 1, "x is NULL"),
            ((FAKE, 1, 2, 64, None, OTHER), 1, "xq"), ((FAKE, 1, 2, 64, OUT, None), 1, "xs"),
            ((FAKE + 2, 1, 2, 64, OUT, OTHER), 4, "x is"), ((FAKE, 1, 2, 64, OUT, OTHER + 4), 4, "xs"),
            ((FAKE, 1, 2, 64, FAKE + 16, OTHER), 1, "overlaps"), ((FAKE, 1, 2, 64, OUT, OUT + 16), 1, "overlaps")):
        assert f(*a, None) == status, (a, _err(q))
        assert msg in _err(q), (a, _err(q))


def test_forward_mx_refusals(q):
    def call(d=None, xq=FAKE, xs=FAKE + 4096, M=2, w=None, bias=None, y=OUT, yd=1):
        d = d or q.QDesc.mxfp4(64, 128)
        w = w or q._Weights(OTHER, None, OTHER + 8192, None, None)
        return q.lib.qlinear_forward_mx(ctypes.byref(d.c()), xq, xs, M, ctypes.byref(w), bias, y, yd, None)
    for kw, status, msg in (
            (dict(d=q.QDesc.affine(64, 128)), 3, "MXFP4"), (dict(d=q.QDesc.mxfp4(64, 100)), 2, "32"),
            (dict(M=0), 2, "M must"), (dict(M=(1 << 20) + 1), 3, "2^20"), (dict(yd=3), 1, "y_dtype"),
            (dict(xq=None), 1, "xq"), (dict(xs=None), 1, "xs"), (dict(y=None), 1, "y is"), (dict(y=OUT + 4), 4, "y is"),
            (dict(bias=FAKE + 4), 4, "bias"), (dict(w=q._Weights(OTHER, None, None, None, None)), 1, "scales"),
            (dict(y=FAKE), 1, "overlaps"), (dict(y=OTHER), 1, "overlaps"), (dict(y=FAKE + 4096), 1, "overlaps")):
        assert call(**kw) == status, (kw, _err(q))
        assert msg in _err(q), (kw, _err(q))


def _moe(q, **kw):
    E, K, inner = 4, 128, 96
    a = dict(up=q.QDesc.mxfp4(E * inner, K), down=q.QDesc.mxfp4(E * K, inner), E=E, k=2, x=FAKE, dt=1, M=3,
             r=FAKE + (1 << 20), score=0, norm=1, ids=OUT, wt=OUT + (1 << 20), g=None, u=None, d=None, act=0,
             y=OUT + (1 << 21), yd=1, ws=WS, n=1 << 24) | kw
    w = [a[k] or q._Weights(OTHER + (i << 28), None, OTHER + (i << 28) + (1 << 27), OTHER, OTHER)
         for i, k in enumerate("gud")]
    return q.lib.qmoe_forward(ctypes.byref(a["up"].c()), ctypes.byref(a["down"].c()), a["E"], a["k"], a["x"], a["dt"],
                              a["M"], a["r"], a["score"], a["norm"], a["ids"], a["wt"], ctypes.byref(w[0]),
                              ctypes.byref(w[1]), ctypes.byref(w[2]), a["act"], a["y"], a["yd"], a["ws"], a["n"], None)


def test_moe_refusals(q):
    D = q.QDesc
    for kw, status, msg in (
            (dict(up=D.mxfp4(4 * 96, 100)), 2, "32"), (dict(up=D.q6k(4 * 96, 256)), 3, "4-bit"),
            (dict(down=D.affine(512, 128, 8, 64)), 3, "4-bit"), (dict(down=D.mxfp4(4 * 128, 128)), 2, "down projection"),
            (dict(down=D.mxfp4(4 * 96, 96)), 2, "down projection"), (dict(up=D.mxfp4(4 * 96 + 1, 128)), 2, "multiples"),
            (dict(E=0), 3, "experts"), (dict(E=513), 3, "experts"), (dict(E=3), 2, "multiples"),
            (dict(k=0), 3, "topk"), (dict(k=5), 3, "topk"), (dict(M=0), 2, "M must"), (dict(M=65), 3, "64 tokens"),
            (dict(dt=2), 1, "x_dtype"), (dict(yd=3), 1, "y_dtype"), (dict(score=2), 1, "score"),
            (dict(norm=2), 1, "norm"), (dict(act=2), 1, "activation"), (dict(x=None), 1, "x is NULL"),
            (dict(ids=None), 1, "ids"), (dict(wt=None), 1, "weights"), (dict(y=None), 1, "y is"),
            (dict(r=FAKE + 4), 4, "router"), (dict(ids=OUT + 4), 4, "ids"), (dict(ws=None), 1, "workspace is NULL"),
            (dict(n=16), 1, "too small"), (dict(ws=WS + 8), 4, "workspace"), (dict(y=FAKE), 1, "overlaps"),
            (dict(ws=FAKE), 1, "overlaps"), (dict(ids=OUT + (1 << 20)), 1, "overlaps"), (dict(y=OTHER), 1, "overlaps"),
            (dict(ids=OTHER), 1, "overlaps"), (dict(y=OUT, ids=OUT, r=None), 1, "overlaps"),
            (dict(d=q._Weights(OTHER, None, None, None, None)), 1, "scales"),
            (dict(up=D.mxfp4(1 << 30, 1 << 20), down=D.mxfp4(1 << 22, 1 << 28)), 3, "2^24"),
            (dict(M=64, k=4, up=D.mxfp4(1 << 24, 1 << 10), down=D.mxfp4(1 << 12, 1 << 22)), 3, "2^29")):
        assert _moe(q, **kw) == status, (kw, _err(q))
        assert msg in _err(q), (kw, _err(q))
    n = ctypes.c_size_t(3)
    up, down = D.mxfp4(4 * 96, 128).c(), D.q4k(4 * 128, 256).c()
    f = q.lib.qmoe_workspace_bytes
    assert f(ctypes.byref(up), ctypes.byref(D.mxfp4(512, 96).c()), 3, 4, 2, None) == q.QP_EINVAL
    assert f(ctypes.byref(up), ctypes.byref(down), 3, 4, 2, ctypes.byref(n)) == q.QP_ESHAPE and n.value == 0
    assert f(ctypes.byref(up), ctypes.byref(D.sym4(512, 96).c()), 3, 4, 2, ctypes.byref(n)) == 0 and n.value > 0


def test_binding_refuses(q):
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    up, down = q.QDesc.mxfp4(4 * 96, 128), q.QDesc.mxfp4(512, 96)
    for call in (lambda: q.quantize_activations_mx(x), lambda: q.quantize_activations_mx(x[0]),
                 lambda: q.qlinear_forward_mx(up, x, x, {}), lambda: q.qlinear_forward_mx(up, x[0], x, {}),
                 lambda: q.qmoe_forward(up, down, x, {}, {}, {}, 4, 2, router=x)):
        with pytest.raises(ValueError):
            call()


def test_forward_mx_long_rows(q):
    """Rows whose scales do not fit LDS need whole 128-column steps."""
    w = q._Weights(FAKE, None, FAKE, None, None)
    for M, K in ((5, 95264), (20, 63520), (40, 31264), (3000, 31264), (1, (1 << 20) + 128)):
        assert q.lib.qlinear_forward_mx(ctypes.byref(q.QDesc.mxfp4(8, K).c()), OTHER, WS, M, ctypes.byref(w), None, OUT,
                                        1, None) == q.QP_EUNSUPPORTED and "K % 128" in _err(q), (M, K, _err(q))


def test_selector_by_outputs(q):
    """More rows: the kernels on exact codes while M N <= 2^22, the qGEMM (a workspace for bf16 rows) beyond."""
    n = ctypes.c_size_t(7)
    for M, N, few in ((16, 1 << 20, True), (17, 4096, True), (1024, 4096, True), (1025, 4096, False), (64, 65537, False)):
        assert q.lib.qlinear_workspace_bytes(ctypes.byref(q.QDesc.mxfp4(N, 4096).c()), 1, M, q.QP_KERNEL_AUTO,
                                             ctypes.byref(n)) == 0 and (n.value == 0) == few, (M, N)


def test_longest_rows(q):
    """The longest rows of each format whose metadata fits LDS, and the next."""
    n = ctypes.c_size_t()

    def moe(up, down):
        return q.lib.qmoe_workspace_bytes(ctypes.byref(up.c()), ctypes.byref(down.c()), 64, 1, 1, ctypes.byref(n))
    for make, K, step in ((q.QDesc.mxfp4, 114656, 32), (lambda N, K: q.QDesc.affine(N, K, 4, 32), 28640, 32),
                          (lambda N, K: q.QDesc.affine(N, K, 4, 64), 57280, 64),
                          (lambda N, K: q.QDesc.affine(N, K, 4, 128), 114560, 128), (q.QDesc.q4k, 44800, 256),
                          (lambda N, K: q.QDesc.sym4(N, K, 32), 28640, 32)):
        for k, ok in ((K, True), (K + step, False)):
            assert (moe(make(64, k), q.QDesc.mxfp4(k, 64)) == 0) == ok, (make(64, k), _err(q))
            assert (moe(q.QDesc.mxfp4(k, 64), make(64, k)) == 0) == ok, (make(64, k), _err(q))
    w = q._Weights(FAKE, None, FAKE, None, None)
    for M in (1, 9, 40):
        assert q.lib.qlinear_forward_kernel(ctypes.byref(q.QDesc.mxfp4(8, 114688).c()), FAKE, 1, M, ctypes.byref(w), None,
                                            OUT, 1, q.QP_KERNEL_GEMV, None) == q.QP_EUNSUPPORTED and "long" in _err(q)
