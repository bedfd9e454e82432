"""Workloads of the MLP-block operators around the packed linear layers: RMS norm with residual and int8 output,
8-bit activation checkpoints, the gated pair of projections, and the gradients through packed weights.

Each case names one operator, its sizes and its types.  `run` computes it in plain torch (fp32, or fp64 where values
sit next to a rounding border), or, with `own` set, through this package's entry points."""
import math

import torch

own = False

GROUP = 64          # columns per scale of an 8-bit activation checkpoint
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # decode: one token's residual addition, norm and int8 row in front of an a8w4 projection
        dict(name="norm int8 1x4096", op="norm", M=1, K=4096, dt="bf16", residual=True, q8=True),
        # prefill: the same in 16 bits
        dict(name="norm 2048x8192", op="norm", M=2048, K=8192, dt="bf16", residual=True, q8=False),
        # training: the norm's gradients, joined with the residual stream's gradient
        dict(name="norm bwd 2048x4096", op="norm_bwd", M=2048, K=4096, dt="bf16", q8=False),
        # a short ragged batch whose residual stream was kept in 8 bits, odd row length
        dict(name="norm bwd 77x5121 8-bit", op="norm_bwd", M=77, K=5121, dt="f16", q8=True),
        # the MLP's inner activations of a training batch into 8 bits and back
        dict(name="checkpoint 2048x14336", op="checkpoint", M=2048, K=14336, dt="bf16"),
        # a small ragged one
        dict(name="checkpoint 19x1000", op="checkpoint", M=19, K=1000, dt="f16"),
        # decode of one token through a 4-bit gated block
        dict(name="gated 1x4096x14336 int4", op="gated", M=1, K=4096, N=14336, dt="bf16", fmt="affine", bits=4, gs=64,
             act="silu", save=False),
        # decode of eight sequences through Q4K weights
        dict(name="gated 8x5120x25600 q4k", op="gated", M=8, K=5120, N=25600, dt="bf16", fmt="q4k", bits=4, gs=32,
             act="silu", save=False),
        # a training step's forward, its pre-activations kept in 8 bits
        dict(name="gated 2048x4096x14336 saved", op="gated", M=2048, K=4096, N=14336, dt="bf16", fmt="affine", bits=4,
             gs=64, act="silu", save=True),
        # the same block's backward from those 8 bits
        dict(name="gated bwd 2048x4096x14336", op="gated_bwd", M=2048, K=4096, N=14336, dt="bf16", fmt="affine",
             bits=4, gs=64, act="silu"),
        # the down projection's input gradient
        dict(name="linear bwd 2048x14336x4096", op="linear_bwd", M=2048, K=14336, N=4096, dt="bf16", fmt="affine",
             bits=4, gs=64),
        # a short batch through square Q6K weights
        dict(name="linear bwd 300x8192x8192 q6k", op="linear_bwd", M=300, K=8192, N=8192, dt="bf16", fmt="q6k",
             bits=6, gs=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "checkpoint", "gated", "gated_bwd", "linear_bwd"])
    if op in ("norm", "norm_bwd", "checkpoint"):
        M, K = _log(rng, 1, 4096), _log(rng, 64, 16384)
        if rng.random() < 0.7:
            K = (K + 7) // 8 * 8
        while M * K > 2048 * 8192:
            M = (M + 1) // 2
        c = dict(op=op, M=M, K=K, dt=rng.choice(["bf16", "f16"]))
        if op == "norm":
            c.update(residual=rng.random() < 0.7, q8=rng.random() < 0.5)
        if op == "norm_bwd":
            c.update(q8=rng.random() < 0.5)
        return c
    fmt, bits, gs = rng.choice([("affine", 2, 64), ("affine", 4, 32), ("affine", 4, 64), ("affine", 4, 128),
                                ("affine", 8, 64), ("q4k", 4, 32), ("q6k", 6, 16), ("sym4", 4, 0)])
    K = max(1, _log(rng, 512, 8192) // 256) * 256
    N = _log(rng, 256, 14336)
    if rng.random() < 0.6:
        N = (N + 63) // 64 * 64
    M = _log(rng, 1, 16) if op == "gated" and rng.random() < 0.5 else _log(rng, 17, 2048)
    while M * N * K > 2048 * 4096 * 14336:
        M = (M + 1) // 2
    c = dict(op=op, M=M, K=K, N=N, dt="bf16", fmt=fmt, bits=bits, gs=gs)
    if op == "gated":
        c.update(act=rng.choice(["silu", "gelu_tanh"]), save=M > 16 and rng.random() < 0.6)
    if op == "gated_bwd":
        c.update(act=rng.choice(["silu", "gelu_tanh"]))
    return c


# ---------------------------------------------------------------- packed weights, as include/qlinear.h lays them out
def _pack(u, bits):
    """Codes [N, K] (int64) -> int32 words, least-significant code first."""
    per = 32 // bits
    n, k = u.shape
    w = torch.zeros((n, k // per), dtype=torch.int64, device=u.device)
    for i in range(per):
        w |= u[:, i::per] << (bits * i)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _weights(g, N, K, fmt, bits, gs):
    """Normal weights, quantized per group and packed."""
    W = torch.randn((N, K), generator=g, device="cuda") * 0.02
    none = dict(qweight=None, qweight_hi=None, scales=None, zeros=None, steps=None)
    if fmt == "affine":
        G = W.view(N, K // gs, gs)
        lo, hi = G.amin(-1), G.amax(-1)
        s, b = ((hi - lo) / (2 ** bits - 1)).bfloat16(), lo.bfloat16()
        q = ((G - b.float()[..., None]) / s.float()[..., None]).round().clamp(0, 2 ** bits - 1)
        return dict(none, qweight=_pack(q.view(N, K).long(), bits), scales=s, zeros=b)
    if fmt == "q4k":
        G = W.view(N, K // 32, 32)
        lo, hi = G.amin(-1).clamp(max=0), G.amax(-1).clamp(min=0)
        s = (hi - lo) / 15
        z = -lo / s
        q = ((G - lo[..., None]) / s[..., None]).round().clamp(0, 15)
        sb, zb = s.view(N, K // 256, 8), z.view(N, K // 256, 8)
        st, zt = (sb.amax(-1) / 255).half(), (zb.amax(-1) / 255).half()
        sc = (sb / st.float()[..., None]).round().clamp(0, 255).view(N, K // 32).to(torch.uint8)
        zc = (zb / zt.float()[..., None]).round().clamp(0, 255).view(N, K // 32).to(torch.uint8)
        steps = (st.view(torch.int16).int() & 0xFFFF) | (zt.view(torch.int16).int() << 16)
        return dict(none, qweight=_pack(q.view(N, K).long(), 4), scales=sc, zeros=zc, steps=steps)
    if fmt == "q6k":
        G = W.view(N, K // 16, 16)
        s = G.abs().amax(-1) / 31
        u = (G / s[..., None]).round().clamp(-32, 31).view(N, K).long() + 32
        sb = s.view(N, K // 256, 16)
        st = (sb.amax(-1) / 127).half()
        sc = (sb / st.float()[..., None]).round().clamp(0, 127).view(N, K // 16).to(torch.int8)
        return dict(none, qweight=_pack(u & 15, 4), qweight_hi=_pack(u >> 4, 2), scales=sc, steps=st)
    s = W.abs().amax(-1, keepdim=True) / 7                      # sym4, one scale per output channel
    u = (W / s).round().clamp(-7, 7).long() + 8
    return dict(none, qweight=_pack(u, 4), scales=s)


def _unpack(w, bits):
    """int32 words -> codes (int32) along the last axis."""
    sh = torch.arange(0, 32, bits, device=w.device, dtype=torch.int32)
    return ((w[..., None] >> sh) & (2 ** bits - 1)).flatten(-2)


def _dequant(w, c, dt=torch.float32):
    """The weight matrix [N, K] that packed buffers stand for."""
    N, K, fmt, gs = c["N"], c["K"], c["fmt"], c["gs"]
    q = _unpack(w["qweight"], c["bits"] if fmt == "affine" else 4)
    if fmt == "affine":
        return (q.view(N, K // gs, gs).to(dt) * w["scales"].to(dt)[..., None] + w["zeros"].to(dt)[..., None]).view(N, K)
    if fmt == "q4k":
        st = (w["steps"] & 0xFFFF).to(torch.int16).view(torch.float16).to(dt)
        zt = (w["steps"] >> 16).to(torch.int16).view(torch.float16).to(dt)
        s = w["scales"].to(dt).view(N, K // 256, 8) * st[..., None]
        z = w["zeros"].to(dt).view(N, K // 256, 8) * zt[..., None]
        return ((q.view(N, K // 256, 8, 32).to(dt) - z[..., None]) * s[..., None]).view(N, K)
    if fmt == "q6k":
        q = (q | (_unpack(w["qweight_hi"], 2) << 4)) - 32
        s = w["scales"].to(dt).view(N, K // 256, 16) * w["steps"].to(dt)[..., None]
        return (q.view(N, K // 256, 16, 16).to(dt) * s[..., None]).view(N, K)
    return (q - 8).to(dt) * w["scales"].to(dt)


# ---------------------------------------------------------------- inputs
def _activations(g, M, K, dt, scale=1.0):
    """Normal values with a few large columns, as residual streams have them."""
    x = torch.randn((M, K), generator=g, device="cuda") * scale
    big = torch.randint(0, K, (max(1, K // 512),), generator=g, device="cuda")
    x[:, big] *= 10
    return x.to(dt)


def _checkpoint(x):
    """int8 codes [M, K] and fp32 scales [M, ceil(K / GROUP)] of x."""
    M, K = x.shape
    n = -(-K // GROUP)
    G = torch.nn.functional.pad(x.float(), (0, n * GROUP - K)).view(M, n, GROUP)
    s = (G.abs().amax(-1).double() / 127).float()
    q = (G.double() / s.double()[..., None]).nan_to_num(0).round().clamp(-127, 127)
    return q.view(M, -1)[:, :K].to(torch.int8).contiguous(), s


def _restore(q, s, dt=torch.float32):
    K = q.shape[1]
    return q.to(dt) * s.to(dt).repeat_interleave(GROUP, 1)[:, :K]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    op, M, K, dt = c["op"], c["M"], c["K"], DT[c["dt"]]
    t = dict(case=c, plan={})
    if op in ("norm", "norm_bwd"):
        t["weight"] = (1 + 0.1 * torch.randn(K, generator=g, device="cuda")).to(dt)
        if op == "norm":
            t["x"] = _activations(g, M, K, dt, 0.5)
            t["residual"] = _activations(g, M, K, dt) if c["residual"] else None
        else:
            s = _activations(g, M, K, dt)
            t["rstd"] = (s.double().square().mean(-1) + EPS).rsqrt().float()
            t["s"], t["s_saved"] = (None, _checkpoint(s)) if c["q8"] else (s, None)
            t["dy"] = (torch.randn((M, K), generator=g, device="cuda") * 1e-2).to(dt)
            t["ds_in"] = (torch.randn((M, K), generator=g, device="cuda") * 1e-2).to(dt)
    elif op == "checkpoint":
        t["x"] = _activations(g, M, K, dt)
    else:
        N = c["N"]
        t["w"] = _weights(g, N, K, c["fmt"], c["bits"], c["gs"])
        if op != "linear_bwd":
            t["w2"] = _weights(g, N, K, c["fmt"], c["bits"], c["gs"])
        if op == "gated":
            t["x"] = _activations(g, M, K, dt)
        else:
            t["dy"] = (torch.randn((M, N), generator=g, device="cuda") * 1e-2).to(dt)
        if op == "gated_bwd":
            t["gate"] = _checkpoint(torch.randn((M, N), generator=g, device="cuda") * 1.3)
            t["up"] = _checkpoint(torch.randn((M, N), generator=g, device="cuda") * 1.3)
    return t


# ---------------------------------------------------------------- one pass
def _act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    a = math.sqrt(2 / math.pi)
    th = torch.tanh(a * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * a * (1 + 3 * 0.044715 * g * g)


def run(state):
    if own:
        return _own(state)
    t, c = state, state["case"]
    op, dt = c["op"], DT[c["dt"]]
    if op == "norm":
        s = t["x"] if t["residual"] is None else (t["x"].float() + t["residual"].float()).to(dt)
        out = {} if t["residual"] is None else {"s": s}
        if not c["q8"]:
            f = s.float()
            r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
            return dict(out, y=(f * r * t["weight"].float()).to(dt))
        d = s.double()
        y = d * torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS) * t["weight"].double()
        ys = (y.abs().amax(-1, keepdim=True) / 127).float()
        return dict(out, y=(y / ys.double()).nan_to_num(0).round().clamp(-127, 127).float() * ys)
    if op == "norm_bwd":
        s = t["s"].float() if t["s"] is not None else _restore(*t["s_saved"])
        dy, w, r = t["dy"].float(), t["weight"].float(), t["rstd"][:, None]
        xh, wdy = s * r, dy * w
        ds = r * (wdy - xh * (wdy * xh).mean(-1, keepdim=True)) + t["ds_in"].float()
        return {"ds": ds.to(dt), "dweight": (dy * xh).sum(0)}
    if op == "checkpoint":
        return {"x": _restore(*_checkpoint(t["x"])).to(dt)}
    if op == "gated":
        x = t["x"].float()
        g, u = x @ _dequant(t["w"], c).t(), x @ _dequant(t["w2"], c).t()
        out = {"h": (_act(g, c["act"])[0] * u).to(dt)}
        if c["save"]:
            out.update(gate=_restore(*_checkpoint(g)).to(dt), up=_restore(*_checkpoint(u)).to(dt))
        return out
    dy = t["dy"].float()
    if op == "linear_bwd":
        return {"dx": (dy @ _dequant(t["w"], c)).to(dt)}
    g, u = _restore(*t["gate"]), _restore(*t["up"])
    a, da = _act(g, c["act"])
    dg, du = dy * u * da, dy * a
    return {"dgate": dg.to(dt), "dup": du.to(dt),
            "dx": (dg @ _dequant(t["w"], c) + du @ _dequant(t["w2"], c)).to(dt)}


def _desc(q, c):
    if c["fmt"] == "affine":
        return q.QDesc.affine(c["N"], c["K"], c["bits"], c["gs"], "bf16")
    return {"q4k": q.QDesc.q4k, "q6k": q.QDesc.q6k, "sym4": q.QDesc.sym4}[c["fmt"]](c["N"], c["K"])


def _own(t):
    from bit_weight_only_qlinear_amd import qlinear as q
    c = t["case"]
    op, dt = c["op"], c["dt"]
    if op == "norm":
        o = q.qnorm_forward(t["x"], t["weight"], residual=t["residual"], eps=EPS, quantize=c["q8"])
        out = {} if t["residual"] is None else {"s": o.s}
        return dict(out, y=o.yq * o.ys[:, None] if c["q8"] else o.y)
    if op == "norm_bwd":
        ds, dw = q.qnorm_backward(t["dy"], t["s"], t["rstd"], t["weight"], saved=t["s_saved"], ds_in=t["ds_in"])
        return {"ds": ds, "dweight": dw}
    if op == "checkpoint":
        return {"x": q.qpack_checkpoint_restore(q.qpack_checkpoint(t["x"]), dt)}
    d = _desc(q, c)
    if op == "gated":
        o = q.qlinear_gated_forward(d, t["x"], t["w"], t["w2"], act=c["act"], save=c["save"])
        if not c["save"]:
            return {"h": o.h}
        return {"h": o.h, "gate": q.qpack_checkpoint_restore(o.gate, dt), "up": q.qpack_checkpoint_restore(o.up, dt)}
    if op == "linear_bwd":
        return {"dx": q.qlinear_backward(d, t["dy"], t["w"])}
    o = q.qlinear_gated_backward(d, t["dy"], t["w"], t["w2"], t["gate"], t["up"], act=c["act"])
    return {"dgate": o.dgate, "dup": o.dup, "dx": o.dx}


# ---------------------------------------------------------------- what a pass cannot do without
def _weight_bytes(c):
    N, K = c["N"], c["K"]
    if c["fmt"] == "affine":
        return N * K * c["bits"] // 8 + 4 * N * (K // c["gs"])
    if c["fmt"] == "q4k":
        return N * K // 2 + N * K // 16 + N * K // 64
    if c["fmt"] == "q6k":
        return N * K * 3 // 4 + N * K // 16 + N * K // 128
    return N * K // 2 + 4 * N


def work(case):
    c = case
    op, M, K = c["op"], c["M"], c["K"]
    saved = lambda n: M * n + 4 * M * -(-n // GROUP)  # noqa: E731  bytes of an 8-bit checkpoint
    if op == "norm":
        out = M * K + 4 * M if c["q8"] else 2 * M * K
        return {"bytes": M * K * (6 if c["residual"] else 2) + out + 2 * K, "flops": 5 * M * K}
    if op == "norm_bwd":
        return {"bytes": M * K * 6 + (saved(K) if c["q8"] else 2 * M * K) + 4 * M + 6 * K, "flops": 10 * M * K}
    if op == "checkpoint":
        return {"bytes": 4 * M * K + 2 * saved(K), "flops": 4 * M * K}
    N = c["N"]
    if op == "gated":
        return {"bytes": 2 * _weight_bytes(c) + 2 * M * (K + N) + (2 * saved(N) if c["save"] else 0),
                "flops": 4 * M * N * K + 6 * M * N}
    if op == "linear_bwd":
        return {"bytes": _weight_bytes(c) + 2 * M * (K + N), "flops": 2 * M * N * K}
    return {"bytes": 2 * _weight_bytes(c) + 2 * saved(N) + 2 * M * (K + 3 * N), "flops": 4 * M * N * K + 12 * M * N}


# ---------------------------------------------------------------- the definition in 64 bits
def _products(a, w, c, transpose):
    """a [M, .] times the weight matrix (transposed where `transpose`), 1024 weight rows at a time."""
    N, out = c["N"], []
    acc = torch.zeros((a.shape[0], c["K"]), dtype=torch.float64, device="cuda")
    for lo in range(0, N, 1024):
        hi = min(N, lo + 1024)
        part = {k: None if v is None else v[lo:hi] for k, v in w.items()}
        W = _dequant(part, dict(c, N=hi - lo), torch.float64)
        if transpose:
            out.append(torch.mm(a, W.t()))
        else:
            acc += torch.mm(a[:, lo:hi], W)
    return torch.cat(out, 1) if transpose else acc


def _saved(x):
    """What a checkpoint of x (64 bits) stands for."""
    out = x.clone()
    for lo in range(0, x.shape[1], GROUP):
        part = x[:, lo:lo + GROUP]
        step = (part.abs().max(-1, keepdim=True).values / 127).float().double()
        out[:, lo:lo + GROUP] = torch.where(step > 0, torch.round(part / step), 0 * part) * step
    return out


def exact(case, seed):
    """The definition in 64 bits."""
    t, c = prepare(case, seed), dict(case)
    op = c["op"]
    f = lambda v: v.to(torch.float64)  # noqa: E731
    if op == "norm":
        s = f(t["x"]) + (0 if t["residual"] is None else f(t["residual"]))
        s = f(s.to(DT[c["dt"]]))                 # the stream is kept in its type, and normed as it is kept
        y = s / (s.pow(2).sum(-1, keepdim=True) / c["K"] + EPS).sqrt() * f(t["weight"])
        if c["q8"]:
            step = f((y.abs().max(-1, keepdim=True).values / 127).float())
            y = torch.where(step > 0, torch.round(y / step), 0 * y) * step
        return {"y": y} if t["residual"] is None else {"s": s, "y": y}
    if op == "norm_bwd":
        r, dy = f(t["rstd"])[:, None], f(t["dy"])
        s = f(t["s"]) if t["s"] is not None else _restore(*t["s_saved"], torch.float64)
        gw = dy * f(t["weight"])
        dot = (gw * s).sum(-1, keepdim=True) / c["K"]
        return {"ds": gw * r - s * dot * r.pow(3) + f(t["ds_in"]), "dweight": (dy * s * r).sum(0)}
    if op == "checkpoint":
        return {"x": _saved(f(t["x"]))}
    if op == "linear_bwd":
        return {"dx": _products(f(t["dy"]), t["w"], c, False)}
    if op == "gated":
        g, u = _products(f(t["x"]), t["w"], c, True), _products(f(t["x"]), t["w2"], c, True)
    else:
        g, u = _restore(*t["gate"], torch.float64), _restore(*t["up"], torch.float64)
    if c["act"] == "silu":
        sig = torch.sigmoid(g)
        a, da = g * sig, sig + g * sig * (1 - sig)
    else:
        k = math.sqrt(2 / math.pi)
        v = torch.tanh(k * (g + 0.044715 * g ** 3))
        a, da = g * (1 + v) / 2, (1 + v) / 2 + g * (1 - v ** 2) * k * (1 + 0.134145 * g ** 2) / 2
    if op == "gated":
        return {"h": a * u, "gate": _saved(g), "up": _saved(u)} if c["save"] else {"h": a * u}
    dg, du = f(t["dy"]) * u * da, f(t["dy"]) * a
    return {"dgate": dg, "dup": du, "dx": _products(dg, t["w"], c, False) + _products(du, t["w2"], c, False)}
