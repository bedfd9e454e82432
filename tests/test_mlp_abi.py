"""Argument checks of the MLP-block entry points: every refusal happens on
the host, before any launch (CPU; the addresses are never read)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

FAKE, OUT, OTHER = 1 << 20, 1 << 21, 1 << 22


@pytest.fixture(scope="module")
def q():
    from bit_weight_only_qlinear_amd import qlinear
    return qlinear


def _err(q):
    return q.lib.qpack_last_error().decode()


def _w(q):
    return q._Weights(FAKE, FAKE, FAKE, FAKE, FAKE)


def _norm(q, **kw):
    a = dict(x=FAKE, r=OTHER, dt=1, M=2, K=64, w=None, eps=1e-6, s=OUT, y=OUT + 4096, yq=None,
             ys=None, rstd=None) | kw
    return q.lib.qnorm_forward(a["x"], a["r"], a["dt"], a["M"], a["K"], a["w"], a["eps"], a["s"],
                               a["y"], a["yq"], a["ys"], a["rstd"], None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(dt=2), 1, "x_dtype"), (dict(M=0), 2, "positive"), (dict(K=0), 2, "positive"),
    (dict(M=(1 << 21) + 1), 3, "2^21"), (dict(K=(1 << 24) + 8), 3, "2^24"),
    (dict(M=1 << 20, K=1 << 15), 3, "2^34"), (dict(M=1 << 20, K=2049), 3, "2^31"),
    (dict(eps=0.0), 1, "eps"), (dict(eps=float("inf")), 1, "eps"), (dict(eps=float("nan")), 1, "eps"),
    (dict(y=None), 1, "yq"), (dict(yq=OTHER), 1, "yq"), (dict(y=None, yq=OUT), 1, "yq"),
    (dict(r=None), 1, "residual"), (dict(x=None), 1, "x is NULL"), (dict(x=FAKE + 2), 4, "x is"),
    (dict(r=OTHER + 8), 4, "residual"), (dict(w=FAKE + 2), 4, "weight"), (dict(s=OUT + 8), 4, "s is"),
    (dict(rstd=FAKE + 4), 4, "rstd"), (dict(y=FAKE), 1, "own"), (dict(y=OTHER), 1, "own"),
    (dict(y=OUT), 1, "own"),
])
def test_norm_refusals(q, kw, status, msg):
    assert _norm(q, **kw) == status, _err(q)
    assert msg in _err(q)


def _norm_bwd(q, **kw):
    a = dict(dy=FAKE, s=OTHER, sc=None, ss=None, dt=1, M=2, K=64, w=None, rstd=FAKE, di=None, ds=OUT,
             dw=OUT + 4096, ws=FAKE, n=1 << 20) | kw
    return q.lib.qnorm_backward(a["dy"], a["s"], a["sc"], a["ss"], a["dt"], a["M"], a["K"], a["w"],
                                a["rstd"], a["di"], a["ds"], a["dw"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(dt=2), 1, "x_dtype"), (dict(M=0), 2, "positive"), (dict(s=None), 1, "s_codes"),
    (dict(sc=FAKE), 1, "s_codes"), (dict(s=None, sc=FAKE), 1, "s_codes"),
    (dict(ds=None, dw=None), 1, "both NULL"), (dict(rstd=None), 1, "rstd"),
    (dict(dy=None), 1, "dy"), (dict(ds=OTHER), 1, "must not be"), (dict(ws=None), 1, "workspace"),
    (dict(n=16), 1, "too small"), (dict(ws=FAKE + 4), 4, "workspace"), (dict(dw=FAKE + 4), 4, "dweight"),
])
def test_norm_backward_refusals(q, kw, status, msg):
    assert _norm_bwd(q, **kw) == status, _err(q)
    assert msg in _err(q)


def test_checkpoint_refusals(q):
    c, r = q.lib.qpack_checkpoint, q.lib.qpack_checkpoint_restore
    assert c(FAKE, 2, 2, 64, FAKE, FAKE, None) == q.QP_EINVAL and "x_dtype" in _err(q)
    assert c(FAKE, 1, 0, 64, FAKE, FAKE, None) == q.QP_ESHAPE
    assert c(None, 1, 2, 64, FAKE, FAKE, None) == q.QP_EINVAL
    assert c(FAKE, 1, 2, 64, FAKE + 1, FAKE, None) == q.QP_EALIGN
    assert c(FAKE, 1, 2, 64, FAKE, None, None) == q.QP_EINVAL and "scales" in _err(q)
    assert r(FAKE, FAKE, 2, 64, FAKE, 3, None) == q.QP_EINVAL and "x_dtype" in _err(q)
    assert r(FAKE, FAKE, 2, 0, FAKE, 1, None) == q.QP_ESHAPE
    assert r(FAKE, None, 2, 64, FAKE, 1, None) == q.QP_EINVAL
    assert r(FAKE, FAKE, 2, 64, FAKE + 2, 1, None) == q.QP_EALIGN


def _gated(q, **kw):
    a = dict(d=q.QDesc.affine(64, 512), x=FAKE, dt=1, M=2, bg=None, bu=None, act=0, h=OUT, hdt=1,
             ck=(None,) * 4, ws=None, n=0, g=_w(q), u=_w(q)) | kw
    d = a["d"].c()
    return q.lib.qlinear_gated_forward(ctypes.byref(d), a["x"], a["dt"], a["M"], ctypes.byref(a["g"]),
                                       ctypes.byref(a["u"]), a["bg"], a["bu"], a["act"], a["h"],
                                       a["hdt"], *a["ck"], a["ws"], a["n"], None)


def test_gated_refusals(q):
    D = q.QDesc
    for kw, status, msg in [
        (dict(d=D.affine(64, 500)), 2, "multiple"), (dict(dt=2), 1, "x_dtype"),
        (dict(hdt=3), 1, "h_dtype"), (dict(M=0), 2, "M must"), (dict(M=(1 << 20) + 1), 3, "2^20"),
        (dict(d=D.affine((1 << 26) + 1, 64)), 3, "2^26"), (dict(act=2), 1, "activation"),
        (dict(x=None), 1, "x is NULL"), (dict(h=None), 1, "h is NULL"), (dict(h=FAKE), 1, "own"),
        (dict(h=OUT + 2), 4, "h is"), (dict(bg=FAKE + 2), 4, "bias_gate"), (dict(bu=FAKE + 2), 4, "bias_up"),
        (dict(ck=(FAKE, None, None, None)), 1, "gate_scales"),
        (dict(ck=(FAKE, FAKE, FAKE, None)), 1, "up_scales"),
        (dict(ck=(FAKE, FAKE, FAKE + 4, FAKE)), 4, "up_codes"), (dict(M=17, ws=FAKE + 4, n=1 << 30), 4, "workspace"),
        (dict(M=17), 1, "workspace is NULL"), (dict(M=17, ws=FAKE, n=16), 1, "too small"),
        (dict(ck=(FAKE, FAKE, FAKE, OTHER)), 1, "own"), (dict(ck=(FAKE, FAKE, OTHER, FAKE)), 1, "own"),
        (dict(ck=(FAKE, FAKE, OTHER, OTHER)), 1, "workspace is NULL"), (dict(d=D.affine(64, 96, 4, 32)), 1, "workspace is NULL"),
        (dict(M=1, ck=(FAKE, FAKE, OTHER, OTHER)), 1, "workspace is NULL"),
        (dict(g=q._Weights(FAKE, None, None, FAKE, None)), 1, "scales"),
        (dict(u=q._Weights(FAKE + 4, None, FAKE, FAKE, None)), 4, "qweight"),
    ]:
        assert _gated(q, **kw) == status, (kw, _err(q))
        assert msg in _err(q), (kw, _err(q))


def test_backward_refusals(q):
    d = q.QDesc.affine(64, 512)
    n = ctypes.c_size_t(0)
    size = q.lib.qlinear_backward_workspace_bytes
    assert size(ctypes.byref(d.c()), 2, 0, None) == q.QP_EINVAL
    assert size(ctypes.byref(d.c()), 0, 0, ctypes.byref(n)) == q.QP_ESHAPE
    assert size(ctypes.byref(d.c()), 2, 1, ctypes.byref(n)) == 0 and n.value > 0

    def lin(dy=FAKE, dt=1, M=2, w=None, dx=OUT, xdt=1, ws=FAKE, nb=1 << 30, desc=d):
        w = w or _w(q)
        return q.lib.qlinear_backward(ctypes.byref(desc.c()), dy, dt, M, ctypes.byref(w), dx, xdt, ws,
                                      nb, None)

    def gat(dh=FAKE, dt=1, M=2, act=0, ck=(FAKE,) * 4, dg=None, du=None, dx=OUT, xdt=1, ws=FAKE,
            nb=1 << 30):
        w = _w(q)
        return q.lib.qlinear_gated_backward(ctypes.byref(d.c()), dh, dt, M, ctypes.byref(w),
                                            ctypes.byref(w), act, *ck, dg, du, dx, xdt, ws, nb, None)

    for st, status, msg in [
        (lambda: lin(dt=2), 1, "dy_dtype"), (lambda: lin(xdt=3), 1, "dx_dtype"),
        (lambda: lin(M=-1), 2, "M must"), (lambda: lin(dy=None), 1, "dy"), (lambda: lin(dx=None), 1, "dx"),
        (lambda: lin(dx=OUT + 2), 4, "dx"), (lambda: lin(dx=FAKE), 1, "own"),
        (lambda: lin(ws=None), 1, "workspace"), (lambda: lin(nb=16), 1, "too small"),
        (lambda: lin(w=q._Weights(FAKE, None, None, FAKE, None)), 1, "scales"),
        (lambda: lin(desc=q.QDesc.q4k(8, 300)), 2, "256"),
        (lambda: gat(act=7), 1, "activation"), (lambda: gat(ck=(FAKE, FAKE, None, FAKE)), 1, "up_codes"),
        (lambda: gat(dg=FAKE), 1, "own"), (lambda: gat(du=OUT), 1, "own"),
        (lambda: gat(dg=OTHER, du=OTHER), 1, "own"), (lambda: gat(dg=OTHER + 2), 4, "dgate"),
        (lambda: gat(nb=16), 1, "too small"), (lambda: gat(ws=FAKE + 8), 4, "workspace"),
        (lambda: gat(dt=2), 1, "dh_dtype"),
    ]:
        assert st() == status, (msg, _err(q))
        assert msg in _err(q), (msg, _err(q))


def test_binding_refuses_host_tensors_and_shapes(q):
    """Device, type and shape checks of the binding (host tensors suffice)."""
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    for call in (lambda: q.qnorm_forward(x), lambda: q.qpack_checkpoint(x),
                 lambda: q.qnorm_backward(x, x, torch.zeros(2)),
                 lambda: q.qlinear_gated_forward(q.QDesc.affine(64, 64), x, {}, {}),
                 lambda: q.qlinear_backward(q.QDesc.affine(64, 64), x, {}),
                 lambda: q.qpack_checkpoint_restore((torch.zeros((2, 64), dtype=torch.int8),
                                                     torch.zeros((2, 1))))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        q.qnorm_forward(x[0])
    with pytest.raises(ValueError):
        q.qnorm_backward(x, None, torch.zeros(2))
    with pytest.raises(ValueError):
        q._torch_dt("f64")
    with pytest.raises(ValueError):
        q._act_id("relu")


def test_descriptor_is_copied_and_pickled_after_use(q):
    import copy
    import pickle
    d = q.QDesc.affine(64, 512)
    d._cref, d._buffer_sizes
    for e in (pickle.loads(pickle.dumps(d)), copy.deepcopy(d), copy.copy(d)):
        assert e == d and hash(e) == hash(d) and e._buffer_sizes == d._buffer_sizes
