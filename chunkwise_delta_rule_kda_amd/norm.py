"""The gated norm behind an attention output or between two blocks: binding of
kda_gated_norm (include/kda.h)."""

import ctypes

from . import KdaError, kda_last_error, load_library
from ._tensors import contiguous_like, dtype_code, get_torch, is_tensor, need, on_device, run_on

__all__ = ["kda_gated_norm", "kda_gated_norm_args"]

_P, _I64 = ctypes.c_void_p, ctypes.c_int64


class kda_gated_norm_args(ctypes.Structure):
    _fields_ = (
        [(n, _P) for n in ("x", "gate", "residual", "weight", "next_weight", "out", "next_out")]
        + [(n, _I64) for n in ("M", "G", "D")]
        + [(f"{t}_stride_{d}", _I64) for t in ("x", "gate", "residual") for d in ("m", "g")]
        + [("io_dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("eps", ctypes.c_float),
           ("scale", ctypes.c_float)])


_ACT = {"sigmoid": 0, "silu": 1}


def _rows(t, name):
    """Strides of the rows of t seen as [M, G, D] with G its last axis but one."""
    shape, stride = t.shape, t.stride()
    if t.is_contiguous():  # from the shape: the strides of axes of one entry say nothing
        return (shape[-2] * shape[-1], shape[-1]) if len(shape) > 2 else (shape[-1], 0)
    if not (shape[-1] == 1 or stride[-1] == 1):
        raise KdaError(2, f"the last axis of {name} must be contiguous")
    g = stride[-2] if len(shape) > 2 and shape[-2] > 1 else 0
    m, span = 0, 1  # stride of the collapsed leading axes, rows they span so far
    for n, s in zip(reversed(shape[:-2] if len(shape) > 2 else shape[:-1]),
                    reversed(stride[:-2] if len(shape) > 2 else stride[:-1])):
        if n == 1:
            continue
        if span == 1:
            m = s
        if not (s == m * span):
            raise KdaError(2, f"the leading axes of {name} cannot be seen as one")
        span *= n
    return m, g


def kda_gated_norm(x, gate=None, weight=None, residual=None, *, next_weight=None, eps=1e-6,
                   gate_act="sigmoid", scale=1.0, out=None, next_out=None, stream=None):
    """y = residual + scale * act(gate) * weight * x / sqrt(mean(x^2) + eps) over the last
    axis, in fp32, rounded once; with next_weight (or next_out) also
    z = next_weight * y / sqrt(mean(y^2) + eps) from the unrounded y.

    x: [..., D], bf16 or fp32, D a multiple of 8 up to 16384; e.g. the [B, T, H, 128] output
    of kda_prefill or kda_linear with a norm and a gate for each head, or [B, T, hidden]
    between two blocks. gate, residual: x's shape and dtype, or None. Of these three only
    the last axis has to be contiguous, and the axes before the last two must collapse into
    one (slices of a projection are fine). weight, next_weight: fp32 [D] or None (ones).
    gate_act: "sigmoid" or "silu". out may be x, gate or residual itself where that is
    contiguous. Returns y, or (y, z).
    """
    torch = get_torch()
    is_tensor(x, "x")
    need(x.dim() >= 1, 2, "x must have at least one axis")
    code = dtype_code(x, "x")
    shape, dt = x.shape, x.dtype
    D = shape[-1]
    if not (gate_act in _ACT):
        raise KdaError(4, f"gate_act {gate_act!r} is neither 'sigmoid' nor 'silu'")
    G = shape[-2] if len(shape) > 2 else 1
    if not (D >= 1 and G >= 1):
        raise KdaError(2, f"x has shape {tuple(shape)}")
    M = x.numel() // (D * G)
    st = [0] * 6
    for i, (name, t) in enumerate((("x", x), ("gate", gate), ("residual", residual))):
        if t is None:
            continue
        is_tensor(t, name, dt)
        if not (t.shape == shape):
            raise KdaError(2, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        st[2 * i:2 * i + 2] = _rows(t, name)
    for name, t in (("weight", weight), ("next_weight", next_weight)):
        if t is not None:
            is_tensor(t, name, torch.float32)
            if not (tuple(t.shape) == (D,) and t.is_contiguous()):
                raise KdaError(2, f"{name} must be a contiguous [{D}]")
    for name, t in (("out", out), ("next_out", next_out)):
        if t is not None:
            is_tensor(t, name, dt)
            if not (t.shape == shape and t.is_contiguous()):
                raise KdaError(2, f"{name} must be a contiguous {tuple(shape)}")
    dev = on_device(x, "x gate weight residual next_weight out next_out", gate, weight, residual,
                    next_weight, out, next_out)
    both = next_weight is not None or next_out is not None
    ptr = lambda t: None if t is None else t.data_ptr()
    with run_on(dev, stream) as handle:
        if out is None:
            out = contiguous_like(x)
        if both and next_out is None:
            next_out = contiguous_like(x)
        a = kda_gated_norm_args(ptr(x), ptr(gate), ptr(residual), ptr(weight), ptr(next_weight),
                                ptr(out), ptr(next_out), M, G, D, *st, code, _ACT[gate_act], eps,
                                scale)
        status = load_library().kda_gated_norm(ctypes.byref(a), handle)
    if status:
        raise KdaError(status, kda_last_error())
    return (out, next_out) if both else out
