"""The short causal convolution in front of a recurrence: binding of kda_short_conv
(include/kda.h)."""

import ctypes

from . import KdaError, kda_last_error, load_library
from ._tensors import (channel_strides, contiguous_like, dtype_code, get_torch, is_tensor,
                       new_state, on_device, packer, run_on, sequences, states, vector)

__all__ = ["kda_short_conv", "kda_short_conv_args", "kda_short_conv_check",
           "make_short_conv_args"]

_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32

_ACT = {None: 0, "silu": 1}  # KDA_CONV_SILU


class kda_short_conv_args(ctypes.Structure):
    _fields_ = (
        [(n, _P) for n in ("x", "weight", "bias", "state_in", "cu_seqlens", "out", "state_out")]
        + [(n, _I64) for n in ("B", "T", "C", "W", "N", "x_stride_batch", "x_stride_token")]
        + [(n, _I32) for n in ("io_dtype", "state_dtype", "flags")]
        + [("ssm_state_indices", _P), ("state_out_indices", _P), ("state_pool_slots", _I64),
           ("state_slot_pitch", _I64)])


_pack = packer(kda_short_conv_args)


def _ptr(x):
    return x if x is None or isinstance(x, int) else x.data_ptr()


def make_short_conv_args(*, B, T, C, N, W=4, x_stride=None, **kw):
    """Fill a kda_short_conv_args from raw pointers (ints), tensors or None; the strides
    default to a contiguous x."""
    a = kda_short_conv_args()
    a.B, a.T, a.C, a.W, a.N = B, T, C, W, N
    a.x_stride_batch, a.x_stride_token = x_stride or (T * C, C)
    for name, x in kw.items():
        whole = name in ("io_dtype", "state_dtype", "flags", "state_pool_slots",
                         "state_slot_pitch")
        setattr(a, name, x if whole else _ptr(x))
    return a


def kda_short_conv_check(args):
    """Host-only validation; returns the status code (0 = OK)."""
    return load_library().kda_short_conv_check(ctypes.byref(args))


def kda_short_conv(x, weight, bias=None, state_in=None, cu_seqlens=None, *, activation="silu",
                   output_final_state=True, state_dtype=None, out=None, state_out=None,
                   ssm_state_indices=None, state_out_indices=None, stream=None):
    """Causal convolution of each channel with its own few taps, on the current (or given)
    stream:

        y_t[c] = act(bias[c] + sum_i weight[c, i] x_{t - (W-1) + i}[c]),  i = 0 .. W-1

    in fp32, rounded once. x: [B, T, C], bf16 or fp32, C a multiple of 8; only its last axis
    has to be contiguous (the other strides multiples of 8, the tokens' at most 2^22), so q, k
    and v side by side, or one part of a projection, are taken as they are. weight: fp32 [C, W]
    with W 2, 3 or 4; bias: fp32 [C] or None. Tensors start on multiples of 16 bytes.
    activation: "silu" or None.
    state_in: [N, W - 1, C], the inputs before each sequence, the oldest first, or None
    (zeros); state_out=state_in updates in place. state_dtype: the states' type, bf16 or fp32;
    None is state_in's, or without one x's, in which they are exact. cu_seqlens: int64 [N + 1]
    (B = 1) or None.
    ssm_state_indices (int32 [N]): state_in is a pool [slots, W - 1, C] (its first axis may be
    padded), sequence n starts from slot ssm_state_indices[n] and writes its final state to
    slot state_out_indices[n] (None: the slot it read); the returned state is the pool. Ids
    outside the pool start from zero and write nothing.
    Returns (out, state_out or None).
    """
    torch = get_torch()
    is_tensor(x, "x")
    if x.dim() != 3:
        raise KdaError(2, "x must have three axes, [B, T, channels]")
    B, T, C = x.shape
    io, dt = dtype_code(x, "x"), x.dtype
    is_tensor(weight, "weight", torch.float32)
    if weight.dim() != 2 or weight.shape[0] != C or not weight.is_contiguous():
        raise KdaError(2, f"weight must be a contiguous [{C}, taps]")
    W = weight.shape[1]
    if not 2 <= W <= 4:
        raise KdaError(2, f"weight has {W} taps, 2 to 4 are supported")
    vector(bias, "bias", C)
    if activation not in _ACT:
        raise KdaError(4, f"activation {activation!r} is neither 'silu' nor None")
    xb, xt = channel_strides(x, "x", B, T)
    N = sequences(cu_seqlens, B)
    state_out, state_dtype, st, slots, pitch = states(
        state_in, state_out, state_dtype, dt, N, W - 1, C, ssm_state_indices, state_out_indices)
    if out is not None:
        is_tensor(out, "out")
        if not (out.shape == x.shape and out.dtype == dt and out.is_contiguous()):
            raise KdaError(2, f"out must be a contiguous {tuple(x.shape)} of {dt}")
    dev = on_device(x, "x weight bias state_in cu_seqlens out state_out ssm_state_indices "
                    "state_out_indices", weight, bias, state_in, cu_seqlens, out, state_out,
                    ssm_state_indices, state_out_indices)
    with run_on(dev, stream) as handle:
        if out is None:
            out = contiguous_like(x)
        if state_out is None and output_final_state:
            state_out = new_state(x, state_in, (N, W - 1, C), state_dtype)
        a = _pack(
            *[0 if t is None else t.data_ptr() for t in (
                x, weight, bias, state_in, cu_seqlens, out, state_out)],
            B, T, C, W, N, xb, xt, io, st, _ACT[activation],
            0 if ssm_state_indices is None else ssm_state_indices.data_ptr(),
            0 if state_out_indices is None else state_out_indices.data_ptr(), slots, pitch)
        status = load_library().kda_short_conv(a, handle)
    if status:
        raise KdaError(status, kda_last_error())
    return out, state_out
