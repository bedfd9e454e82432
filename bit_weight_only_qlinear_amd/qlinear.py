"""Thin ctypes binding of libqlinear (include/qlinear.h).

Argument marshalling only: torch supplies device memory and the current HIP
stream; every step of the computation runs in the library's HIP kernels.
The library must be built (``python -m bit_weight_only_qlinear_amd.build``
or ``__graft_entry__.build()``); importing this module without it raises.
"""
import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Any, NamedTuple, Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlinear.so")

QP_OK, QP_EINVAL, QP_ESHAPE, QP_EUNSUPPORTED, QP_EALIGN, QP_EHIP = range(6)
QP_FMT_AFFINE, QP_FMT_Q4K, QP_FMT_Q6K, QP_FMT_SYM4, QP_FMT_MXFP4 = range(5)
QP_F16, QP_BF16, QP_F32 = range(3)
QP_ACT_SILU, QP_ACT_GELU_TANH = range(2)
QP_SCORE_SOFTMAX, QP_SCORE_SIGMOID = range(2)
QP_CHECKPOINT_GROUP = 64
QP_KERNEL_AUTO, QP_KERNEL_GEMV, QP_KERNEL_GEMM, QP_KERNEL_GEMV_MFMA = range(4)

FMT_IDS = {"affine": QP_FMT_AFFINE, "q4k": QP_FMT_Q4K, "q6k": QP_FMT_Q6K,
           "sym4": QP_FMT_SYM4, "mxfp4": QP_FMT_MXFP4}
DTYPE_IDS = {"f16": QP_F16, "bf16": QP_BF16, "f32": QP_F32}
ACT_IDS = {"silu": QP_ACT_SILU, "gelu_tanh": QP_ACT_GELU_TANH}
SCORE_IDS = {"softmax": QP_SCORE_SOFTMAX, "sigmoid": QP_SCORE_SIGMOID}
BUFFERS = ("qweight", "qweight_hi", "scales", "zeros", "steps")


class QLinearError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"qlinear status {status}: {message}")
        self.status = status


class _Desc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("super_block", ctypes.c_int32),
                ("meta_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class _Weights(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in BUFFERS]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build the HIP library first "
            "(python -m bit_weight_only_qlinear_amd.build)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    D, W = ctypes.POINTER(_Desc), ctypes.POINTER(_Weights)
    sig = {
        "qpack_abi_version": (I32, []),
        "qpack_last_error": (ctypes.c_char_p, []),
        "qpack_sizes": (I32, [D, ctypes.POINTER(ctypes.c_size_t)]),
        "qpack_quantize": (I32, [D, P, W, P]),
        "qpack_quantize_hqq": (I32, [D, P, W, I32, ctypes.c_float, ctypes.c_float,
                                     ctypes.c_float, P]),
        "qpack_unpack_codes": (I32, [D, W, P, P]),
        "qpack_pack_codes": (I32, [D, P, W, P]),
        "qpack_dequantize": (I32, [D, W, P, I32, P]),
        "qlinear_forward": (I32, [D, P, I32, I64, W, P, P, I32, P]),
        "qlinear_forward_kernel": (I32, [D, P, I32, I64, W, P, P, I32, I32, P]),
        "qlinear_workspace_bytes": (I32, [D, I32, I64, I32, ctypes.POINTER(ctypes.c_size_t)]),
        "qlinear_forward_ws": (I32, [D, P, I32, I64, W, P, P, I32, I32, P, ctypes.c_size_t, P]),
        "qlinear_forward_static": (I32, [D, P, I32, I64, W, P, P, I32, I32, P]),
        "qpack_encode_nested": (I32, [D, P, P, W, P, P]),
        "qpack_concat_n": (I32, [D, I32, D, W, W, P]),
        "qpack_quantize_activations": (I32, [P, I32, I64, I64, P, P, P]),
        "qlinear_forward_a8w4": (I32, [D, P, P, I64, W, P, P, I32, P]),
        "qnorm_forward": (I32, [P, P, I32, I64, I64, P, ctypes.c_float, P, P, P, P, P, P]),
        "qnorm_backward_workspace_bytes": (I32, [I64, I64, ctypes.POINTER(ctypes.c_size_t)]),
        "qnorm_backward": (I32, [P, P, P, P, I32, I64, I64, P, P, P, P, P, P, ctypes.c_size_t, P]),
        "qpack_checkpoint": (I32, [P, I32, I64, I64, P, P, P]),
        "qpack_checkpoint_restore": (I32, [P, P, I64, I64, P, I32, P]),
        "qlinear_gated_workspace_bytes": (I32, [D, I64, I32, ctypes.POINTER(ctypes.c_size_t)]),
        "qlinear_gated_forward": (I32, [D, P, I32, I64, W, W, P, P, I32, P, I32, P, P, P, P, P,
                                        ctypes.c_size_t, P]),
        "qlinear_backward_workspace_bytes": (I32, [D, I64, I32, ctypes.POINTER(ctypes.c_size_t)]),
        "qlinear_backward": (I32, [D, P, I32, I64, W, P, I32, P, ctypes.c_size_t, P]),
        "qlinear_gated_backward": (I32, [D, P, I32, I64, W, W, I32, P, P, P, P, P, P, P, I32, P,
                                         ctypes.c_size_t, P]),
        "qpack_quantize_activations_mx": (I32, [P, I32, I64, I64, P, P, P]),
        "qlinear_forward_mx": (I32, [D, P, P, I64, W, P, P, I32, P]),
        "qmoe_workspace_bytes": (I32, [D, D, I64, I32, I32, ctypes.POINTER(ctypes.c_size_t)]),
        "qmoe_forward": (I32, [D, D, I32, I32, P, I32, I64, P, I32, I32, P, P, W, W, W, I32, P, I32, P,
                               ctypes.c_size_t, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()
EXPORTED = ("qpack_abi_version", "qpack_last_error", "qpack_sizes", "qpack_quantize",
            "qpack_quantize_hqq",
            "qpack_unpack_codes", "qpack_pack_codes", "qpack_dequantize",
            "qlinear_forward", "qlinear_forward_kernel", "qlinear_workspace_bytes",
            "qlinear_forward_ws", "qlinear_forward_static", "qpack_encode_nested",
            "qpack_concat_n",
            "qpack_quantize_activations",
            "qlinear_forward_a8w4",
            "qnorm_forward", "qnorm_backward_workspace_bytes", "qnorm_backward",
            "qpack_checkpoint", "qpack_checkpoint_restore",
            "qlinear_gated_workspace_bytes", "qlinear_gated_forward",
            "qlinear_backward_workspace_bytes", "qlinear_backward", "qlinear_gated_backward",
            "qpack_quantize_activations_mx", "qlinear_forward_mx", "qmoe_workspace_bytes",
            "qmoe_forward")


@dataclass(frozen=True)
class QDesc:
    """Python form of qp_desc."""
    fmt: str
    bits: int
    group_size: int
    N: int
    K: int
    meta: str = "bf16"          # affine metadata dtype
    super_block: int = 0

    @staticmethod
    def affine(N, K, bits=4, group_size=64, meta="bf16"):
        return QDesc("affine", bits, group_size, N, K, meta, 0)

    @staticmethod
    def q4k(N, K):
        return QDesc("q4k", 4, 32, N, K, "f16", 256)

    @staticmethod
    def q6k(N, K):
        return QDesc("q6k", 6, 16, N, K, "f16", 256)

    @staticmethod
    def sym4(N, K, group_size=None):
        return QDesc("sym4", 4, K if group_size is None else group_size, N, K, "f32", 0)

    @staticmethod
    def mxfp4(N, K):
        return QDesc("mxfp4", 4, 32, N, K, "f16", 0)

    @functools.cached_property
    def _cref(self):
        """The C form, built once (read only)."""
        return ctypes.byref(self.c())

    @functools.cached_property
    def _buffer_sizes(self):
        """(name, bytes) of every buffer, from the library."""
        return tuple(qpack_sizes(self).items())

    def __getstate__(self):   # the cached C form stays with the process
        return {k: v for k, v in self.__dict__.items() if not k.startswith("_")}

    def c(self):
        return _Desc(FMT_IDS[self.fmt], self.bits, self.group_size, self.super_block,
                     DTYPE_IDS[self.meta], 0, self.N, self.K)


def _check(status):
    if status != QP_OK:
        raise QLinearError(status, lib.qpack_last_error().decode())


def _stream(device=None):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def qpack_sizes(desc: QDesc):
    out = (ctypes.c_size_t * 5)()
    d = desc.c()
    _check(lib.qpack_sizes(ctypes.byref(d), out))
    return dict(zip(BUFFERS, [int(v) for v in out]))


def _buf_dtypes(desc):
    import torch
    meta = {"f16": torch.float16, "bf16": torch.bfloat16}.get(desc.meta, torch.float16)
    if desc.fmt == "affine":
        return dict(qweight=torch.int32, scales=meta, zeros=meta)
    if desc.fmt == "q4k":
        return dict(qweight=torch.int32, scales=torch.uint8, zeros=torch.uint8,
                    steps=torch.int32)
    if desc.fmt == "q6k":
        return dict(qweight=torch.int32, qweight_hi=torch.int32, scales=torch.int8,
                    steps=torch.float16)
    if desc.fmt == "mxfp4":
        return dict(qweight=torch.int32, scales=torch.uint8)
    return dict(qweight=torch.int32, scales=torch.float32)


def alloc_weights(desc: QDesc, device="cuda"):
    """Empty device buffers of the sizes qpack_sizes gives (torch memory)."""
    import torch
    sizes = qpack_sizes(desc)
    dts = _buf_dtypes(desc)
    out = {}
    for name in BUFFERS:
        if sizes[name]:
            dt = dts[name]
            itemsize = torch.empty(0, dtype=dt).element_size()
            # allocated to the next multiple of 16 bytes (the library reads
            # its buffers in 16-byte units); the view has the exact size
            padded = (sizes[name] + 15) // 16 * 16
            out[name] = torch.empty(padded // itemsize, dtype=dt,
                                    device=device)[: sizes[name] // itemsize]
        else:
            out[name] = None
    return out


def _wstruct(w):
    return _Weights(*[None if w.get(n) is None else w[n].data_ptr() for n in BUFFERS])


def qpack_quantize(desc: QDesc, W, out=None):
    """W: device fp32 [N, K] -> dict of packed buffers (torch tensors)."""
    if out is None:
        out = alloc_weights(desc, W.device)
    d, ws = desc.c(), _wstruct(out)
    _check(lib.qpack_quantize(ctypes.byref(d), _ptr(W), ctypes.byref(ws), _stream(W.device)))
    return out


def qpack_quantize_hqq(desc: QDesc, W, out=None, iters=20, lp_norm=0.7, beta=10.0,
                       kappa=1.01):
    """AFFINE only: W device fp32 [N, K] -> packed buffers, with the HQQ zero
    point per group (see qpack_quantize_hqq in include/qlinear.h)."""
    if out is None:
        out = alloc_weights(desc, W.device)
    d, ws = desc.c(), _wstruct(out)
    _check(lib.qpack_quantize_hqq(ctypes.byref(d), _ptr(W), ctypes.byref(ws), int(iters),
                                  float(lp_norm), float(beta), float(kappa),
                                  _stream(W.device)))
    return out


def qpack_unpack_codes(desc: QDesc, w, codes=None):
    import torch
    if codes is None:
        dt = torch.int8 if desc.fmt in ("q6k", "sym4") else torch.uint8
        codes = torch.empty((desc.N, desc.K), dtype=dt, device=w["qweight"].device)
    d, ws = desc.c(), _wstruct(w)
    _check(lib.qpack_unpack_codes(ctypes.byref(d), ctypes.byref(ws), _ptr(codes),
                                  _stream(codes.device)))
    return codes


def qpack_pack_codes(desc: QDesc, codes, out=None):
    if out is None:
        out = alloc_weights(desc, codes.device)
    d, ws = desc.c(), _wstruct(out)
    _check(lib.qpack_pack_codes(ctypes.byref(d), _ptr(codes), ctypes.byref(ws),
                                _stream(codes.device)))
    return out


def qpack_dequantize(desc: QDesc, w, out_dtype="f32", out=None):
    import torch
    tdt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[out_dtype]
    if out is None:
        out = torch.empty((desc.N, desc.K), dtype=tdt, device=w["qweight"].device)
    d, ws = desc.c(), _wstruct(w)
    _check(lib.qpack_dequantize(ctypes.byref(d), ctypes.byref(ws), _ptr(out),
                                DTYPE_IDS[out_dtype], _stream(out.device)))
    return out


def _xdtype(t):
    import torch
    if t.dtype == torch.float16:
        return "f16"
    if t.dtype == torch.bfloat16:
        return "bf16"
    raise TypeError(f"activations must be float16 or bfloat16, got {t.dtype}")


def workspace_bytes(desc: QDesc, M: int, x_dtype: str = "bf16",
                    kernel: int = QP_KERNEL_AUTO) -> int:
    """Device workspace bytes qlinear_forward can use (qlinear_workspace_bytes)."""
    d, n = desc.c(), ctypes.c_size_t(0)
    _check(lib.qlinear_workspace_bytes(ctypes.byref(d), DTYPE_IDS[x_dtype], M, kernel,
                                       ctypes.byref(n)))
    return n.value


def qlinear_forward(desc: QDesc, x, w, bias=None, y_dtype: Optional[str] = None,
                    kernel: int = QP_KERNEL_AUTO, out=None, workspace="auto"):
    """y [M, N] = x [M, K] W^T (+ bias).  x: fp16/bf16 device tensor.

    workspace: "auto" allocates what the call can use from torch's caching
    allocator on the current stream; None runs without one; or a device
    tensor (its bytes are the workspace)."""
    import torch
    xd = _xdtype(x)
    yd = y_dtype or xd
    tdt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[yd]
    M = x.shape[0]
    if out is None:
        out = torch.empty((M, desc.N), dtype=tdt, device=x.device)
    buf, nbytes = None, 0
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto', None or a tensor, got {workspace!r}")
        nbytes = workspace_bytes(desc, M, xd, kernel)
        if nbytes:
            buf = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    elif workspace is not None:
        buf, nbytes = workspace, workspace.numel() * workspace.element_size()
    d, ws = desc.c(), _wstruct(w)
    _check(lib.qlinear_forward_ws(ctypes.byref(d), _ptr(x), DTYPE_IDS[xd], M,
                                  ctypes.byref(ws), _ptr(bias), _ptr(out), DTYPE_IDS[yd],
                                  kernel, _ptr(buf), nbytes, _stream(x.device)))
    return out


def qlinear_forward_static(desc: QDesc, x, w, out, bias=None, kernel: int = QP_KERNEL_AUTO):
    """qlinear_forward_static: the forward into the caller's `out` (its dtype
    is the output dtype) with the library's static scratch in place of a
    workspace; the C call allocates nothing."""
    import torch
    yd = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}[out.dtype]
    d, ws = desc.c(), _wstruct(w)
    _check(lib.qlinear_forward_static(ctypes.byref(d), _ptr(x), DTYPE_IDS[_xdtype(x)], x.shape[0],
                                      ctypes.byref(ws), _ptr(bias), _ptr(out), DTYPE_IDS[yd],
                                      kernel, _stream(x.device)))
    return out


def concat_n(descs, weights):
    """Stack layers of one format and K along N (qpack_concat_n): returns
    (QDesc of the stacked layer, its buffers)."""
    import dataclasses
    d0 = descs[0]
    dout = dataclasses.replace(d0, N=sum(d.N for d in descs))
    out = alloc_weights(dout, device=weights[0]["qweight"].device)
    n = len(descs)
    dins = (_Desc * n)(*[d.c() for d in descs])
    wins = (_Weights * n)(*[_wstruct(w) for w in weights])
    _check(lib.qpack_concat_n(ctypes.byref(dout.c()), n, dins, wins, ctypes.byref(_wstruct(out)),
                              _stream(weights[0]["qweight"].device)))
    return dout, out


def convert_to_nested(desc: QDesc, codes, s, z=None):
    """Plain int4 (codes uint8 [N, K], s, z fp32 [N, K/32]) or int6 (codes
    int8 [N, K], s fp32 [N, K/16]) -> nested Q4K / Q6K buffers with the codes
    unchanged (qpack_pack_codes + qpack_encode_nested).  Returns (buffers,
    bad) with bad a device int32 that is 1 if any input was invalid."""
    import torch
    w = alloc_weights(desc, device=codes.device)
    _check(lib.qpack_pack_codes(ctypes.byref(desc.c()), _ptr(codes), ctypes.byref(_wstruct(w)),
                                _stream(codes.device)))
    bad = torch.zeros(4, dtype=torch.int32, device=codes.device)
    _check(lib.qpack_encode_nested(ctypes.byref(desc.c()), _ptr(s), _ptr(z),
                                   ctypes.byref(_wstruct(w)), _ptr(bad), _stream(codes.device)))
    return w, bad


def quantize_activations(x):
    """Per-token symmetric int8 activations (qpack_quantize_activations):
    x fp16/bf16 [M, K] -> (xq int8 [M, K], xs fp32 [M])."""
    import torch
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    _check(lib.qpack_quantize_activations(_ptr(x), DTYPE_IDS[_xdtype(x)], M, K, _ptr(xq),
                                          _ptr(xs), _stream(x.device)))
    return xq, xs


def qlinear_forward_a8w4(desc: QDesc, xq, xs, w, bias=None, y_dtype: str = "bf16", out=None):
    """y [M, N] = xs[m] * s_n * sum_k xq[m, k] q[n, k] (+ bias fp32 [N]) for
    SYM4 weights with one scale per output channel."""
    import torch
    tdt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[y_dtype]
    M = xq.shape[0]
    if out is None:
        out = torch.empty((M, desc.N), dtype=tdt, device=xq.device)
    d, ws = desc.c(), _wstruct(w)
    _check(lib.qlinear_forward_a8w4(ctypes.byref(d), _ptr(xq), _ptr(xs), M, ctypes.byref(ws),
                                    _ptr(bias), _ptr(out), DTYPE_IDS[y_dtype],
                                    _stream(xq.device)))
    return out


# ---- the MLP block around the packed layers: RMS norm, 8-bit activation
# checkpoints, the gated pair of projections, and input gradients.  Every
# tensor is checked before the call: device, type, shape, contiguous rows.

class QNorm(NamedTuple):
    """qnorm_forward's outputs; the ones that were not asked for are None."""
    y: Any        # [M, K] of x's type, or None where quantized
    s: Any        # the residual stream x + residual (x itself without one)
    rstd: Any     # fp32 [M]
    yq: Any       # int8 [M, K] and
    ys: Any       # fp32 [M]: quantize=True


class QGated(NamedTuple):
    """qlinear_gated_forward's outputs: h, and the checkpoints (codes, scales)
    of both pre-activations where they were asked for."""
    h: Any
    gate: Any
    up: Any


class QGatedGrads(NamedTuple):
    """qlinear_gated_backward's outputs."""
    dx: Any
    dgate: Any
    dup: Any


def _torch_dt(name):
    import torch
    if name not in DTYPE_IDS:
        raise ValueError(f"dtype must be one of {tuple(DTYPE_IDS)}, got {name!r}")
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _arg(t, name, shape, dtype, device):
    """Address of a device tensor argument of the given shape and type, rows
    packed."""
    if t.device == device and t.dtype == dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _opt(t, name, shape, dtype, device):
    return None if t is None else _arg(t, name, shape, dtype, device)


def _rows(t, name):
    """(M, K, dtype name) of an activation matrix."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix [M, K], got {t.dim()} dimensions")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor, got {t.device}")
    return t.shape[0], t.shape[1], _xdtype(t)


def _weights_arg(desc, w, name, device):
    """The weight struct, its buffers checked against the descriptor."""
    ptrs = []
    for n, need in desc._buffer_sizes:
        t = w.get(n) if need else None
        if need and (t is None or t.device != device or not t.is_contiguous() or t.nbytes < need):
            raise ValueError(f"{name}[{n!r}] must be a contiguous tensor of {need} bytes on {device}")
        ptrs.append(t.data_ptr() if need else None)
    return ctypes.byref(_Weights(*ptrs))


def _run(device, fn, *args):
    """Calls a library function on the device's current stream (appended as
    the last argument), with that device current."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # without a Stream object
    stream = raw(device.index) if raw else torch.cuda.current_stream(device).cuda_stream
    if torch.cuda.current_device() == device.index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status != QP_OK:
        _check(status)


def _scratch(nbytes, device):
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _groups(n):
    return (n + QP_CHECKPOINT_GROUP - 1) // QP_CHECKPOINT_GROUP


def qnorm_forward(x, weight=None, residual=None, eps: float = 1e-6, quantize: bool = False,
                  need_rstd: bool = False, s_out=None) -> QNorm:
    """RMS norm of s = x + residual, times weight: 16-bit rows, or with
    `quantize` int8 rows with one scale each (qlinear_forward_a8w4's
    activations).  x, residual [M, K] and weight [K]: fp16 or bf16.  s goes
    into `s_out` where given (x or residual itself: in place)."""
    import torch
    M, K, xd = _rows(x, "x")
    dev, dt = x.device, x.dtype
    px = _arg(x, "x", (M, K), dt, dev)
    pr = _opt(residual, "residual", (M, K), dt, dev)
    pw = _opt(weight, "weight", (K,), dt, dev)
    s, ps = x, None
    if residual is not None:
        s = torch.empty_like(x) if s_out is None else s_out
        ps = _arg(s, "s_out", (M, K), dt, dev)
    elif s_out is not None:
        raise ValueError("s_out needs a residual (s is x without one)")
    y = yq = ys = rstd = None
    if quantize:
        yq = torch.empty((M, K), dtype=torch.int8, device=dev)
        ys = torch.empty((M,), dtype=torch.float32, device=dev)
    else:
        y = torch.empty_like(x)
    if need_rstd:
        rstd = torch.empty((M,), dtype=torch.float32, device=dev)
    p = [None if t is None else t.data_ptr() for t in (y, yq, ys, rstd)]
    _run(dev, lib.qnorm_forward, px, pr, DTYPE_IDS[xd], M, K, pw, eps, ps, *p)
    return QNorm(y, s, rstd, yq, ys)


def qnorm_backward(dy, s, rstd, weight=None, saved=None, ds_in=None, need_ds: bool = True,
                   need_dweight: bool = True):
    """Gradients of qnorm_forward's 16-bit output: (ds [M, K], dweight fp32
    [K]), None for one that is not needed.  s: the forward's stream, or None
    with `saved`, its checkpoint (codes, scales).  ds is the gradient of x
    and of the residual; ds_in is added to it."""
    import torch
    M, K, xd = _rows(dy, "dy")
    dev, dt = dy.device, dy.dtype
    if (s is None) == (saved is None):
        raise ValueError("pass s, or its checkpoint as saved")
    codes, scales = (None, None) if saved is None else saved
    ps = _opt(s, "s", (M, K), dt, dev)
    pc = _opt(codes, "saved codes", (M, K), torch.int8, dev)
    psc = _opt(scales, "saved scales", (M, _groups(K)), torch.float32, dev)
    args = (_arg(dy, "dy", (M, K), dt, dev), ps, pc, psc, DTYPE_IDS[xd], M, K,
            _opt(weight, "weight", (K,), dt, dev), _arg(rstd, "rstd", (M,), torch.float32, dev),
            _opt(ds_in, "ds_in", (M, K), dt, dev))
    ds = torch.empty_like(dy) if need_ds else None
    dw = torch.empty((K,), dtype=torch.float32, device=dev) if need_dweight else None
    ws, n = None, 0
    if need_dweight:
        size = ctypes.c_size_t(0)
        _check(lib.qnorm_backward_workspace_bytes(M, K, ctypes.byref(size)))
        n = size.value
        ws = _scratch(n, dev)
    _run(dev, lib.qnorm_backward, *args, *[None if t is None else t.data_ptr()
                                           for t in (ds, dw, ws)], n)
    return ds, dw


def qpack_checkpoint(x):
    """8-bit checkpoint of activations x [M, K]: (codes int8 [M, K], scales
    fp32 [M, ceil(K / 64)])."""
    import torch
    M, K, xd = _rows(x, "x")
    px = _arg(x, "x", (M, K), x.dtype, x.device)
    codes = torch.empty((M, K), dtype=torch.int8, device=x.device)
    scales = torch.empty((M, _groups(K)), dtype=torch.float32, device=x.device)
    _run(x.device, lib.qpack_checkpoint, px, DTYPE_IDS[xd], M, K, codes.data_ptr(),
         scales.data_ptr())
    return codes, scales


def qpack_checkpoint_restore(saved, dtype: str = "bf16"):
    """The values a checkpoint (codes, scales) stands for, [M, K] of `dtype`."""
    import torch
    codes, scales = saved
    if codes.dim() != 2:
        raise ValueError("codes must be a matrix [M, K]")
    M, K = codes.shape
    if not codes.is_cuda:
        raise ValueError(f"codes must be a GPU tensor, got {codes.device}")
    pc = _arg(codes, "codes", (M, K), torch.int8, codes.device)
    ps = _arg(scales, "scales", (M, _groups(K)), torch.float32, codes.device)
    x = torch.empty((M, K), dtype=_torch_dt(dtype), device=codes.device)
    _run(codes.device, lib.qpack_checkpoint_restore, pc, ps, M, K, x.data_ptr(), DTYPE_IDS[dtype])
    return x


def _act_id(act):
    if act not in ACT_IDS:
        raise ValueError(f"act must be one of {tuple(ACT_IDS)}, got {act!r}")
    return ACT_IDS[act]


def qlinear_gated_forward(desc: QDesc, x, gate, up, act: str = "silu", bias_gate=None,
                          bias_up=None, h_dtype: Optional[str] = None,
                          save: bool = False) -> QGated:
    """h [M, N] = act(x Wg^T + bias_gate) * (x Wu^T + bias_up) for two packed
    layers of one descriptor; with `save` also the 8-bit checkpoints of both
    pre-activations for qlinear_gated_backward.  (16 rows and fewer then leave
    the exact-code kernels for the fp16 product: 46 us in place of 13 for one
    row of an int4 4096 -> 14336 pair.)"""
    import torch
    M, K, xd = _rows(x, "x")
    dev, N = x.device, desc.N
    px = _arg(x, "x", (M, desc.K), x.dtype, dev)
    wg, wu = _weights_arg(desc, gate, "gate", dev), _weights_arg(desc, up, "up", dev)
    pb = [_opt(b, n, (N,), x.dtype, dev) for b, n in ((bias_gate, "bias_gate"), (bias_up, "bias_up"))]
    hd = h_dtype or xd
    a = _act_id(act)
    h = torch.empty((M, N), dtype=_torch_dt(hd), device=dev)
    ck = [None] * 4
    if save:
        ck = [torch.empty((M, N), dtype=torch.int8, device=dev),
              torch.empty((M, _groups(N)), dtype=torch.float32, device=dev),
              torch.empty((M, N), dtype=torch.int8, device=dev),
              torch.empty((M, _groups(N)), dtype=torch.float32, device=dev)]
    size = ctypes.c_size_t(0)
    _check(lib.qlinear_gated_workspace_bytes(desc._cref, M, int(save), ctypes.byref(size)))
    ws = _scratch(size.value, dev) if size.value else None
    _run(dev, lib.qlinear_gated_forward, desc._cref, px, DTYPE_IDS[xd], M, wg, wu, *pb, a,
         h.data_ptr(), DTYPE_IDS[hd],
         *[None if t is None else t.data_ptr() for t in (*ck, ws)], size.value)
    return QGated(h, tuple(ck[:2]) if save else None, tuple(ck[2:]) if save else None)


def _backward_workspace(desc, M, gated, device):
    size = ctypes.c_size_t(0)
    _check(lib.qlinear_backward_workspace_bytes(desc._cref, M, int(gated), ctypes.byref(size)))
    return _scratch(size.value, device), size.value


def qlinear_backward(desc: QDesc, dy, w, dx_dtype: Optional[str] = None):
    """dx [M, K] = dy [M, N] W: the input gradient of qlinear_forward."""
    import torch
    M, _, yd = _rows(dy, "dy")
    dev = dy.device
    py = _arg(dy, "dy", (M, desc.N), dy.dtype, dev)
    ww = _weights_arg(desc, w, "w", dev)
    xd = dx_dtype or yd
    dx = torch.empty((M, desc.K), dtype=_torch_dt(xd), device=dev)
    ws, n = _backward_workspace(desc, M, False, dev)
    _run(dev, lib.qlinear_backward, desc._cref, py, DTYPE_IDS[yd], M, ww, dx.data_ptr(), DTYPE_IDS[xd], ws.data_ptr(), n)
    return dx


def qlinear_gated_backward(desc: QDesc, dh, gate, up, gate_saved, up_saved, act: str = "silu",
                           need_dpre: bool = True, dx_dtype: Optional[str] = None) -> QGatedGrads:
    """Backward of qlinear_gated_forward from its checkpoints: dx, and with
    `need_dpre` the gradients of both projections' outputs."""
    import torch
    M, _, yd = _rows(dh, "dh")
    dev, N = dh.device, desc.N
    ph = _arg(dh, "dh", (M, N), dh.dtype, dev)
    wg, wu = _weights_arg(desc, gate, "gate", dev), _weights_arg(desc, up, "up", dev)
    pk = []
    for (codes, scales), n in ((gate_saved, "gate_saved"), (up_saved, "up_saved")):
        pk += [_arg(codes, n + " codes", (M, N), torch.int8, dev),
               _arg(scales, n + " scales", (M, _groups(N)), torch.float32, dev)]
    a = _act_id(act)
    xd = dx_dtype or yd
    dx = torch.empty((M, desc.K), dtype=_torch_dt(xd), device=dev)
    dg, du = (torch.empty_like(dh), torch.empty_like(dh)) if need_dpre else (None, None)
    ws, n = _backward_workspace(desc, M, True, dev)
    _run(dev, lib.qlinear_gated_backward, desc._cref, ph, DTYPE_IDS[yd], M, wg, wu, a, *pk,
         *[None if t is None else t.data_ptr() for t in (dg, du)], dx.data_ptr(), DTYPE_IDS[xd],
         ws.data_ptr(), n)
    return QGatedGrads(dx, dg, du)


# ---- MXFP4 activations, and mixture-of-experts layers for few tokens

class QMoE(NamedTuple):
    """qmoe_forward's outputs: y [M, K], and the experts (int32 [M, topk])
    and their weights (fp32 [M, topk]) of each token."""
    y: Any
    ids: Any
    weights: Any


def quantize_activations_mx(x):
    """MXFP4 rows of x [M, K] (fp16, bf16 or fp32, K % 32 == 0): (codes int32
    [M, K / 8], scales uint8 [M, K / 32])."""
    import torch
    if x.dim() != 2:
        raise ValueError(f"x must be a matrix [M, K], got {x.dim()} dimensions")
    if not x.is_cuda:
        raise ValueError(f"x must be a GPU tensor, got {x.device}")
    xd = "f32" if x.dtype == torch.float32 else _xdtype(x)
    M, K = x.shape
    px = _arg(x, "x", (M, K), x.dtype, x.device)
    xq = torch.empty((M, K // 8), dtype=torch.int32, device=x.device)
    xs = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device)
    _run(x.device, lib.qpack_quantize_activations_mx, px, DTYPE_IDS[xd], M, K, xq.data_ptr(), xs.data_ptr())
    return xq, xs


def qlinear_forward_mx(desc: QDesc, xq, xs, w, bias=None, y_dtype: str = "bf16", out=None):
    """y [M, N] = X W^T (+ bias fp32 [N]) for MXFP4 activations (codes and
    scales of quantize_activations_mx) and MXFP4 weights."""
    import torch
    if xq.dim() != 2:
        raise ValueError(f"xq must be a matrix [M, K / 8], got {xq.dim()} dimensions")
    if not xq.is_cuda:
        raise ValueError(f"xq must be a GPU tensor, got {xq.device}")
    M, dev = xq.shape[0], xq.device
    pq = _arg(xq, "xq", (M, desc.K // 8), torch.int32, dev)
    ps = _arg(xs, "xs", (M, desc.K // 32), torch.uint8, dev)
    ww = _weights_arg(desc, w, "w", dev)
    pb = _opt(bias, "bias", (desc.N,), torch.float32, dev)
    tdt = _torch_dt(y_dtype)
    if out is None:
        out = torch.empty((M, desc.N), dtype=tdt, device=dev)
    po = _arg(out, "out", (M, desc.N), tdt, dev)
    _run(dev, lib.qlinear_forward_mx, desc._cref, pq, ps, M, ww, pb, po, DTYPE_IDS[y_dtype])
    return out


def qmoe_forward(desc_up: QDesc, desc_down: QDesc, x, gate, up, down, experts: int, topk: int, router=None,
                 ids=None, weights=None, score: str = "softmax", norm: bool = True, act: str = "silu",
                 y_dtype: Optional[str] = None) -> QMoE:
    """A mixture-of-experts layer for up to 64 tokens x [M, K]: the experts'
    packed layers stacked along N (gate and up of desc_up, down of desc_down).
    Pass the router's weights [experts, K], or each token's ids (int32
    [M, topk]) and weights (fp32 [M, topk])."""
    import torch
    M, K, xd = _rows(x, "x")
    dev = x.device
    if (router is None) != (ids is not None and weights is not None) or (ids is None) != (weights is None):
        raise ValueError("pass router, or ids and weights")
    if score not in SCORE_IDS:
        raise ValueError(f"score must be one of {tuple(SCORE_IDS)}, got {score!r}")
    px = _arg(x, "x", (M, desc_up.K), x.dtype, dev)
    pr = _opt(router, "router", (experts, desc_up.K), x.dtype, dev)
    if router is None:
        pi = _arg(ids, "ids", (M, topk), torch.int32, dev)
        pw = _arg(weights, "weights", (M, topk), torch.float32, dev)
    wg, wu = _weights_arg(desc_up, gate, "gate", dev), _weights_arg(desc_up, up, "up", dev)
    wd = _weights_arg(desc_down, down, "down", dev)
    a, yd = _act_id(act), y_dtype or xd
    size = ctypes.c_size_t(0)
    _check(lib.qmoe_workspace_bytes(desc_up._cref, desc_down._cref, M, experts, topk, ctypes.byref(size)))
    if router is not None:
        ids = torch.empty((M, topk), dtype=torch.int32, device=dev)
        weights = torch.empty((M, topk), dtype=torch.float32, device=dev)
        pi, pw = ids.data_ptr(), weights.data_ptr()
    y = torch.empty((M, K), dtype=_torch_dt(yd), device=dev)
    ws = _scratch(size.value, dev)
    _run(dev, lib.qmoe_forward, desc_up._cref, desc_down._cref, experts, topk, px, DTYPE_IDS[xd], M, pr,
         SCORE_IDS[score], int(norm), pi, pw, wg, wu, wd, a, y.data_ptr(), DTYPE_IDS[yd], ws.data_ptr(),
         size.value)
    return QMoE(y, ids, weights)
