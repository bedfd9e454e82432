"""Workloads of the microscaled 4-bit format (MXFP4: E2M1 codes, one power-of-two scale per 32 columns) and of
mixture-of-experts layers for a few tokens.

Each case names one operator, its sizes and its types.  `run` computes it in plain torch (fp32, router logits in
fp64), or, with `own` set, through this package's entry points."""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 32          # columns per scale


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # decode: one token's activations in front of a 4-bit x 4-bit projection
        dict(name="quantize 1x4096", op="quantize", M=1, K=4096, dt="bf16"),
        # prefill: an MLP's inner activations in front of the down projection
        dict(name="quantize 2048x14336", op="quantize", M=2048, K=14336, dt="bf16"),
        # decode of one token, 16-bit activations
        dict(name="linear 1x4096x14336", op="linear", M=1, K=4096, N=14336, dt="bf16"),
        # decode of a ragged batch of sequences
        dict(name="linear 13x8192x8192 f16", op="linear", M=13, K=8192, N=8192, dt="f16"),
        # prefill and training forward
        dict(name="linear 2048x4096x14336", op="linear", M=2048, K=4096, N=14336, dt="bf16"),
        # decode of sixteen sequences with both operands in 4 bits
        dict(name="mx x mx 16x5120x25600", op="mxmx", M=16, K=5120, N=25600, dt="bf16"),
        # prefill with both operands in 4 bits
        dict(name="mx x mx 2048x4096x14336", op="mxmx", M=2048, K=4096, N=14336, dt="bf16"),
        # training around frozen weights: the down projection's input gradient
        dict(name="linear bwd 2048x14336x4096", op="linear_bwd", M=2048, K=14336, N=4096, dt="bf16"),
        # a short batch through square weights
        dict(name="linear bwd 300x8192x8192 f16", op="linear_bwd", M=300, K=8192, N=8192, dt="f16"),
        # one token through a layer of few large experts, 4-bit affine weights
        dict(name="moe 1x4096x14336 2 of 8 int4", op="moe", M=1, K=4096, I=14336, E=8, topk=2, dt="bf16", fmt="affine",
             gs=64, act="silu", score="softmax", norm=True),
        # sixteen sequences through a layer of many small experts
        dict(name="moe 16x2048x1024 8 of 64", op="moe", M=16, K=2048, I=1024, E=64, topk=8, dt="bf16", fmt="mxfp4",
             gs=32, act="silu", score="softmax", norm=False),
        # a ragged batch that reaches almost every expert
        dict(name="moe 50x4096x1536 4 of 32 f16", op="moe", M=50, K=4096, I=1536, E=32, topk=4, dt="f16", fmt="mxfp4",
             gs=32, act="gelu_tanh", score="sigmoid", norm=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "mxmx", "linear_bwd", "moe", "moe"])
    dt = rng.choice(["bf16", "bf16", "f16"])
    if op == "quantize":
        M, K = _log(rng, 1, 4096), _log(rng, 2, 512) * BLOCK
        while M * K > 2048 * 14336:
            M = (M + 1) // 2
        return dict(op=op, M=M, K=K, dt=rng.choice(["bf16", "f16", "f32"]))
    if op == "moe":
        E = _log(rng, 2, 128)
        topk = min(E, _log(rng, 1, 8))
        fmt, gs = rng.choice([("mxfp4", 32), ("mxfp4", 32), ("affine", 32), ("affine", 64), ("affine", 128)])
        step = max(gs, 32)
        K, inner = _log(rng, 512, 4096) // step * step, _log(rng, 256, 14336) // step * step
        while E * K * inner > 8 * 4096 * 14336:
            inner = max(step, inner // 2 // step * step)
        return dict(op=op, M=_log(rng, 1, 64), K=K, I=inner, E=E, topk=topk, dt=dt, fmt=fmt, gs=gs,
                    act=rng.choice(["silu", "gelu_tanh"]), score=rng.choice(["softmax", "sigmoid"]),
                    norm=rng.random() < 0.5)
    K, N = _log(rng, 16, 448) * BLOCK, _log(rng, 256, 25600)
    if rng.random() < 0.6:
        K, N = (K + 127) // 128 * 128, (N + 63) // 64 * 64
    M = _log(rng, 1, 16) if op != "linear_bwd" and rng.random() < 0.5 else _log(rng, 17, 2048)
    while M * N * K > 2048 * 4096 * 14336:
        M = (M + 1) // 2
    return dict(op=op, M=M, K=K, N=N, dt=dt)


# ---------------------------------------------------------------- packed weights, as include/qlinear.h lays them out
def _pack(u):
    """4-bit codes [N, K] (int64) -> int32 words, least-significant code first."""
    n, k = u.shape
    w = torch.zeros((n, k // 8), dtype=torch.int64, device=u.device)
    for i in range(8):
        w |= u[:, i::8] << (4 * i)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _unpack(w):
    sh = torch.arange(0, 32, 4, device=w.device, dtype=torch.int32)
    return ((w[..., None] >> sh) & 15).flatten(-2)


def _mx_codes(x):
    """E2M1 codes (sign in bit 3) and E8M0 scale bytes of x: per 32 columns the scale 2^(floor(log2 max) - 2), the
    codes the nearest values, ties to the even code, 6 at most."""
    M, K = x.shape
    G = x.float().view(M, K // BLOCK, BLOCK)
    top = G.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1].int() - 3, -127).clamp(min=-127)
    a = torch.ldexp(G.abs(), -e[..., None])
    c = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() +
         (a >= 3.5).int() + (a > 5).int())
    return (c + 8 * (G < 0).int()).view(M, K), (e + 127).to(torch.uint8)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mx_values(codes, scales):
    t = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    M, K = codes.shape
    v = t[codes.long()].view(M, K // BLOCK, BLOCK)
    return torch.ldexp(v, scales.int()[..., None] - 127).view(M, K)


def _weights(g, N, K, fmt, gs):
    """Normal weights, quantized and packed."""
    none = dict(qweight=None, qweight_hi=None, scales=None, zeros=None, steps=None)
    parts = []
    rows = max(1, (1 << 26) // K)
    for lo in range(0, N, rows):
        W = torch.randn((min(rows, N - lo), K), generator=g, device="cuda") * 0.02
        if fmt == "mxfp4":
            c, s = _mx_codes(W)
            parts.append((_pack(c.long()), s, None))
        else:
            G = W.view(-1, K // gs, gs)
            lo_, hi = G.amin(-1), G.amax(-1)
            s, b = ((hi - lo_) / 15).bfloat16(), lo_.bfloat16()
            q = ((G - b.float()[..., None]) / s.float()[..., None]).round().clamp(0, 15)
            parts.append((_pack(q.view(-1, K).long()), s, b))
    q, s, b = (None if p[0] is None else torch.cat(p) for p in zip(*parts))
    return dict(none, qweight=q, scales=s, zeros=b)


def _dequant(w, K, fmt, gs):
    """The fp32 weight matrix that packed buffers stand for."""
    q = _unpack(w["qweight"])
    if fmt == "mxfp4":
        return _mx_values(q, w["scales"])
    return (q.view(-1, K // gs, gs).float() * w["scales"].float()[..., None] + w["zeros"].float()[..., None]).view(-1, K)


def _expert(w, e, rows):
    return {k: None if v is None else v[e * rows:(e + 1) * rows] for k, v in w.items()}


# ---------------------------------------------------------------- inputs
def _activations(g, M, K, dt, scale=1.0):
    """Normal values with a few large columns, as residual streams have them."""
    x = torch.randn((M, K), generator=g, device="cuda") * scale
    big = torch.randint(0, K, (max(1, K // 512),), generator=g, device="cuda")
    x[:, big] *= 10
    return x.to(dt)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    op, M, K, dt = c["op"], c["M"], c["K"], DT[c["dt"]]
    t = dict(case=c)
    if op == "quantize":
        t["x"] = _activations(g, M, K, dt, 0.02 if c["dt"] == "f32" else 1.0)
    elif op == "moe":
        E, inner = c["E"], c["I"]
        t["x"] = _activations(g, M, K, dt)
        t["router"] = (torch.randn((E, K), generator=g, device="cuda") / math.sqrt(K)).to(dt)
        t["gate"] = _weights(g, E * inner, K, c["fmt"], c["gs"])
        t["up"] = _weights(g, E * inner, K, c["fmt"], c["gs"])
        t["down"] = _weights(g, E * K, inner, c["fmt"], c["gs"])
    else:
        N = c["N"]
        t["w"] = _weights(g, N, K, "mxfp4", 32)
        t["x"] = ((torch.randn((M, N), generator=g, device="cuda") * 1e-2).to(dt) if op == "linear_bwd"
                  else _activations(g, M, K, dt))
    return t


# ---------------------------------------------------------------- one pass
def _act(v, kind):
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))


def _route(x, router, c):
    """Experts [M, topk] by falling score (ties: the lower index) and their weights.  Logits in fp64: the choice sits
    next to a border."""
    logits = x.double() @ router.double().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, top = order.indices[:, :c["topk"]], order.values[:, :c["topk"]]
    if c["score"] == "sigmoid":
        w = 1 / (1 + torch.exp(-top))
    else:
        hi = order.values[:, :1]
        w = torch.exp(top - hi) / torch.exp(logits - hi).sum(1, keepdim=True)
    if c["norm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.int(), w.float()


def run(state):
    if own:
        return _own(state)
    t, c = state, state["case"]
    op, dt, K = c["op"], DT[c["dt"]], c["K"]
    if op == "quantize":
        return {"x": _mx_values(*_mx_codes(t["x"])).bfloat16()}
    if op == "linear":
        return {"y": (t["x"].float() @ _dequant(t["w"], K, "mxfp4", 32).t()).to(dt)}
    if op == "mxmx":
        return {"y": (_mx_values(*_mx_codes(t["x"])) @ _dequant(t["w"], K, "mxfp4", 32).t()).to(dt)}
    if op == "linear_bwd":
        return {"dx": (t["x"].float() @ _dequant(t["w"], K, "mxfp4", 32)).to(dt)}
    ids, w = _route(t["x"], t["router"], c)
    x, inner, fmt, gs = t["x"].float(), c["I"], c["fmt"], c["gs"]
    y = torch.zeros_like(x)
    for e in range(c["E"]):
        share = (w * (ids == e)).sum(1, keepdim=True)
        gate = x @ _dequant(_expert(t["gate"], e, inner), K, fmt, gs).t()
        up = x @ _dequant(_expert(t["up"], e, inner), K, fmt, gs).t()
        y += share * ((_act(gate, c["act"]) * up) @ _dequant(_expert(t["down"], e, K), inner, fmt, gs).t())
    return {"y": y.to(dt), "ids": ids, "weights": w}


def _own(t):
    from bit_weight_only_qlinear_amd import qlinear as q
    c = t["case"]
    op, M, K = c["op"], c["M"], c["K"]
    if op == "quantize":
        d = q.QDesc.mxfp4(M, K)
        if c["dt"] == "f32":
            return {"x": q.qpack_dequantize(d, q.qpack_quantize(d, t["x"]), "bf16")}
        codes, scales = q.quantize_activations_mx(t["x"])
        return {"x": q.qpack_dequantize(d, dict(qweight=codes, scales=scales), "bf16")}
    if op == "moe":
        if c["fmt"] == "mxfp4":
            up, down = q.QDesc.mxfp4(c["E"] * c["I"], K), q.QDesc.mxfp4(c["E"] * K, c["I"])
        else:
            up, down = (q.QDesc.affine(c["E"] * c["I"], K, 4, c["gs"], "bf16"),
                        q.QDesc.affine(c["E"] * K, c["I"], 4, c["gs"], "bf16"))
        o = q.qmoe_forward(up, down, t["x"], t["gate"], t["up"], t["down"], experts=c["E"], topk=c["topk"],
                           router=t["router"], score=c["score"], norm=c["norm"], act=c["act"])
        return {"y": o.y, "ids": o.ids, "weights": o.weights}
    d = q.QDesc.mxfp4(c["N"], K)
    if op == "linear":
        return {"y": q.qlinear_forward(d, t["x"], t["w"])}
    if op == "mxmx":
        codes, scales = q.quantize_activations_mx(t["x"])
        return {"y": q.qlinear_forward_mx(d, codes, scales, t["w"], y_dtype=c["dt"])}
    return {"dx": q.qlinear_backward(d, t["x"], t["w"])}


# ---------------------------------------------------------------- what a pass cannot do without
def _weight_bytes(N, K, fmt, gs):
    return N * K // 2 + (N * K // 32 if fmt == "mxfp4" else 4 * N * (K // gs))


def work(case):
    c = case
    op, M, K = c["op"], c["M"], c["K"]
    if op == "quantize":
        # codes and scales written, and read again for the values
        return {"bytes": M * K * (4 if c["dt"] == "f32" else 2) + 2 * _weight_bytes(M, K, "mxfp4", 32) + 2 * M * K,
                "flops": 4 * M * K}
    if op == "moe":
        E, inner, k = c["E"], c["I"], c["topk"]
        reached = E * (1 - (1 - k / E) ** M)        # experts that some token chooses, on average
        each = 2 * _weight_bytes(inner, K, c["fmt"], c["gs"]) + _weight_bytes(K, inner, c["fmt"], c["gs"])
        return {"bytes": int(reached * each) + 2 * E * K + 4 * M * K + 8 * M * k,
                "flops": 6 * M * k * K * inner + 2 * M * E * K}
    N = c["N"]
    return {"bytes": _weight_bytes(N, K, "mxfp4", 32) + 2 * M * (K + N), "flops": 2 * M * N * K}


# ---------------------------------------------------------------- the definition in 64 bits
def _grid(x):
    """x [M, K] (64 bits) on the format's grid: per 32 columns, with e = floor(log2 max), the multiples of 2^(e - 3)
    below 2^(e - 1), of 2^(e - 2) below 2^e, of 2^(e - 1) above, 6 2^(e - 2) at most."""
    M, K = x.shape
    out = torch.empty_like(x)
    step = max(1, (1 << 24) // M // BLOCK * BLOCK)
    for lo in range(0, K, step):
        g = x[:, lo:lo + step].reshape(M, -1, BLOCK)
        top = g.abs().max(-1, keepdim=True).values
        e = torch.where(top > 0, torch.floor(torch.log2(top)), 0 * top)
        unit = torch.pow(2.0 + 0 * top, e - 3)
        a = g.abs() / unit
        a = torch.where(a < 4, torch.round(a), torch.where(a < 8, 2 * torch.round(a / 2), 4 * torch.round(a / 4)))
        out[:, lo:lo + step] = (torch.sign(g) * a.clamp(max=12) * unit).reshape(M, -1)
    return out


def _matrix(w, K, fmt, gs):
    """Packed rows -> the weight matrix in 64 bits."""
    word = w["qweight"].to(torch.int64) & 0xFFFFFFFF
    q = torch.stack([(word >> (4 * i)) & 15 for i in range(8)], -1).reshape(word.shape[0], K)
    if fmt != "mxfp4":
        s, b = (w[n].to(torch.float64).repeat_interleave(gs, 1) for n in ("scales", "zeros"))
        return q * s + b
    m, e = (q & 1).double(), (q >> 1) & 3
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, e.double() - 1))
    s = torch.pow(2.0, w["scales"].double() - 127).repeat_interleave(BLOCK, 1)
    return torch.where(q >= 8, -v, v) * s


def _product(a, w, K, backward):
    N, out = w["qweight"].shape[0], []
    acc = torch.zeros((a.shape[0], K), dtype=torch.float64, device="cuda")
    for lo in range(0, N, 1024):
        W = _matrix({k: None if v is None else v[lo:lo + 1024] for k, v in w.items()}, K, "mxfp4", 32)
        if backward:
            acc += torch.mm(a[:, lo:lo + 1024], W)
        else:
            out.append(torch.mm(a, W.t()))
    return acc if backward else torch.cat(out, 1)


def exact(case, seed):
    """The definition in 64 bits."""
    t, c = prepare(case, seed), dict(case)
    op, K, x = c["op"], c["K"], t["x"].double()
    if op == "quantize":
        return {"x": _grid(x)}
    if op != "moe":
        return {"dx" if op == "linear_bwd" else "y": _product(_grid(x) if op == "mxmx" else x, t["w"], K,
                                                              op == "linear_bwd")}
    logits = torch.mm(x, t["router"].double().t())
    p = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.softmax(logits, 1)
    # the topk-th largest, again and again, instead of a sort
    left, share, ws = logits.clone(), torch.zeros_like(p), []
    rows = torch.arange(c["M"], device="cuda")
    for _ in range(c["topk"]):
        at = left.argmax(1)
        share[rows, at] = p[rows, at]
        ws.append(p[rows, at])
        left[rows, at] = -math.inf
    total = share.sum(1, keepdim=True) if c["norm"] else 1.0
    share, y = share / total, torch.zeros_like(x)
    for e in range(c["E"]):
        m = (share[:, e] > 0).nonzero()[:, 0]
        if not len(m):
            continue
        g, u = (torch.mm(x[m], _matrix(_expert(t[n], e, c["I"]), K, c["fmt"], c["gs"]).t()) for n in ("gate", "up"))
        if c["act"] == "silu":
            h = g * torch.sigmoid(g) * u
        else:
            h = g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) / 2 * u
        y[m] += share[m, e][:, None] * torch.mm(h, _matrix(_expert(t["down"], e, K), c["I"], c["fmt"], c["gs"]).t())
    return {"y": y, "ids": None, "weights": torch.stack(ws, 1) / total}
