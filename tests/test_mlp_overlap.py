"""Outputs of the MLP-block entry points that reach into another buffer of the
call are refused on the host (CPU; the addresses are never read)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

AT = 1 << 24          # every buffer on a 16 MiB stretch of its own
STEP = 1 << 24


@pytest.fixture(scope="module")
def q():
    if torch.cuda.is_available():
        pytest.skip("host checks: without a GPU, where a call that passed them could not run")
    from bit_weight_only_qlinear_amd import qlinear
    return qlinear


class Call:
    """One call's buffers by name -> (address, bytes), and the call itself."""

    def __init__(self, sizes, run):
        self.at = {n: AT + STEP * i for i, n in enumerate(sizes)}
        self.size, self.run = sizes, run


M, N, K = 40, 64, 512
GROUPS_N, GROUPS_K = 1, 8


def weights(q, p, tag=""):
    return ctypes.byref(q._Weights(p["qweight" + tag], None, p["scales" + tag], p["zeros" + tag], None))


def layer(tag=""):
    return {"qweight" + tag: N * K // 2, "scales" + tag: N * K // 32, "zeros" + tag: N * K // 32}


def calls(q):
    lib, d = q.lib, q.QDesc.affine(N, K, 4, 64, "bf16")._cref
    n = ctypes.c_size_t(0)

    def bytes_of(fn, *a):
        assert fn(*a, ctypes.byref(n)) == 0
        return n.value

    rows = 2 * M * K
    out = {}
    out["norm"] = Call(
        dict(x=rows, residual=rows, weight=2 * K, s=rows, y=rows, rstd=4 * M),
        lambda p: lib.qnorm_forward(p["x"], p["residual"], 1, M, K, p["weight"], 1e-5, p["s"], p["y"], None, None,
                                    p["rstd"], None))
    out["norm int8"] = Call(
        dict(x=rows, residual=rows, weight=2 * K, s=rows, yq=rows // 2, ys=4 * M, rstd=4 * M),
        lambda p: lib.qnorm_forward(p["x"], p["residual"], 1, M, K, p["weight"], 1e-5, p["s"], None, p["yq"], p["ys"],
                                    p["rstd"], None))
    ws = bytes_of(lib.qnorm_backward_workspace_bytes, M, K)
    out["norm backward"] = Call(
        dict(dy=rows, s_codes=rows // 2, s_scales=4 * M * GROUPS_K, weight=2 * K, rstd=4 * M, ds_in=rows, ds=rows,
             dweight=4 * K, workspace=ws),
        lambda p: lib.qnorm_backward(p["dy"], None, p["s_codes"], p["s_scales"], 1, M, K, p["weight"], p["rstd"],
                                     p["ds_in"], p["ds"], p["dweight"], p["workspace"], ws, None))
    out["norm backward, kept"] = Call(
        dict(dy=rows, s=rows, rstd=4 * M, ds=rows),
        lambda p: lib.qnorm_backward(p["dy"], p["s"], None, None, 1, M, K, None, p["rstd"], None, p["ds"], None, None,
                                     0, None))
    out["checkpoint"] = Call(
        dict(x=rows, codes=rows // 2, scales=4 * M * GROUPS_K),
        lambda p: lib.qpack_checkpoint(p["x"], 1, M, K, p["codes"], p["scales"], None))
    out["restore"] = Call(
        dict(codes=rows // 2, scales=4 * M * GROUPS_K, x=2 * rows),
        lambda p: lib.qpack_checkpoint_restore(p["codes"], p["scales"], M, K, p["x"], 2, None))
    wf = bytes_of(lib.qlinear_gated_workspace_bytes, d, M, 1)
    out["gated"] = Call(
        dict(x=rows, bias_gate=2 * N, bias_up=2 * N, h=2 * M * N, gate_codes=M * N, gate_scales=4 * M * GROUPS_N,
             up_codes=M * N, up_scales=4 * M * GROUPS_N, workspace=wf, **layer(), **layer(".up")),
        lambda p: lib.qlinear_gated_forward(d, p["x"], 1, M, weights(q, p), weights(q, p, ".up"), p["bias_gate"],
                                            p["bias_up"], 0, p["h"], 1, p["gate_codes"], p["gate_scales"],
                                            p["up_codes"], p["up_scales"], p["workspace"], wf, None))
    out["gated, few rows"] = Call(
        dict(x=2 * 4 * K, h=4 * 4 * N, **layer(), **layer(".up")),
        lambda p: lib.qlinear_gated_forward(d, p["x"], 1, 4, weights(q, p), weights(q, p, ".up"), None, None, 0,
                                            p["h"], 2, None, None, None, None, None, 0, None))
    wl = bytes_of(lib.qlinear_backward_workspace_bytes, d, M, 0)
    out["linear backward"] = Call(
        dict(dy=2 * M * N, dx=rows, workspace=wl, **layer()),
        lambda p: lib.qlinear_backward(d, p["dy"], 1, M, weights(q, p), p["dx"], 1, p["workspace"], wl, None))
    wb = bytes_of(lib.qlinear_backward_workspace_bytes, d, M, 1)
    out["gated backward"] = Call(
        dict(dh=2 * M * N, gate_codes=M * N, gate_scales=4 * M * GROUPS_N, up_codes=M * N,
             up_scales=4 * M * GROUPS_N, dgate=2 * M * N, dup=2 * M * N, dx=rows, workspace=wb, **layer(),
             **layer(".up")),
        lambda p: lib.qlinear_gated_backward(d, p["dh"], 1, M, weights(q, p), weights(q, p, ".up"), 0,
                                             p["gate_codes"], p["gate_scales"], p["up_codes"], p["up_scales"],
                                             p["dgate"], p["dup"], p["dx"], 1, p["workspace"], wb, None))
    return out


OUTS = {"norm": ("s", "y", "rstd"), "norm int8": ("s", "yq", "ys", "rstd"),
        "norm backward": ("ds", "dweight", "workspace"), "norm backward, kept": ("ds",),
        "checkpoint": ("codes", "scales"), "restore": ("x",),
        "gated": ("h", "gate_codes", "gate_scales", "up_codes", "up_scales", "workspace"),
        "gated, few rows": ("h",), "linear backward": ("dx", "workspace"),
        "gated backward": ("dgate", "dup", "dx", "workspace")}
IN_PLACE = {"norm": (("s", "x"), ("s", "residual")), "norm int8": (("s", "x"), ("s", "residual")),
            "norm backward": (("ds", "dy"), ("ds", "ds_in")), "norm backward, kept": (("ds", "dy"),)}


@pytest.mark.parametrize("name", sorted(OUTS))
def test_outputs_that_reach_into_another_buffer(q, name):
    c = calls(q)[name]
    for o in OUTS[name]:
        for i in c.at:
            if i == o:
                continue
            # the same place; the output's last bytes; its first
            for at in (c.at[i], c.at[i] - c.size[o] + 16, c.at[i] + (c.size[i] - 1) // 16 * 16):
                if at == c.at[i] and (o, i) in IN_PLACE.get(name, ()):
                    continue
                assert c.run(dict(c.at, **{o: at})) == q.QP_EINVAL, (name, o, i, at - c.at[i])
                msg = q.lib.qpack_last_error().decode()
                assert "own" in msg or "must not be" in msg, (name, o, i, msg)


def test_overlap_message_names_both(q):
    c = calls(q)["gated"]
    assert c.run(dict(c.at, h=c.at["up_codes"] + 32)) == q.QP_EINVAL
    msg = q.lib.qpack_last_error().decode()
    assert "h overlaps up_codes" in msg
