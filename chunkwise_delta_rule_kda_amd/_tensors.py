"""What the bindings of the operators beside kda_prefill share: checks of tensors, and the
stream and device a call runs on. These calls can take a few microseconds on the device, so
the checks of the common case are kept short."""

import contextlib
import ctypes
import struct

from . import KDA_BF16, KDA_FP32, KdaError

_torch = _raw_stream = None


def get_torch():
    """The torch module, imported at the first call (the package itself does without)."""
    global _torch, _raw_stream
    if _torch is None:
        import torch

        # the stream's handle without a Stream object around it, where torch has that
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _torch = torch
    return _torch


def need(cond, status, msg):
    if not cond:
        raise KdaError(status, msg)


def dtype_code(t, name):
    dt = t.dtype
    if dt == _torch.bfloat16:
        return KDA_BF16
    if dt == _torch.float32:
        return KDA_FP32
    raise KdaError(3, f"{name} has unsupported dtype {t.dtype}")


def is_tensor(t, name, dtype=None):
    if not isinstance(t, _torch.Tensor):
        raise KdaError(2, f"{name} must be a tensor")
    if dtype is not None and t.dtype != dtype:
        raise KdaError(3, f"{name} is {t.dtype}, expected {dtype}")


def on_device(first, names, *rest):
    """All tensors (or None) are on the first one's CUDA device; names: of all of them."""
    index = first.get_device() if first.is_cuda else -1
    for t in rest:
        if t is not None and t.get_device() != index:
            break
    else:
        if index >= 0:
            return first.device
    for i, t in enumerate((first, *rest)):
        if t is not None and (index < 0 or t.get_device() != index):
            raise KdaError(2, f"{names.split()[i]} must be a CUDA tensor on "
                           f"{first.device if index >= 0 else 'cuda'} (got {t.device})")


def contiguous_like(t):
    """A contiguous uninitialised tensor of t's shape, dtype and device (of a contiguous t
    empty_like is the shortest way there; of another it would keep the strides)."""
    return _torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


@contextlib.contextmanager
def _on(device, stream):
    torch = _torch
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(stream, device=device)
            # what a call allocates belongs to the stream it runs on
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


class _Current:
    """The common case, a call on the current stream of the current device."""

    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return False


def run_on(device, stream):
    """Context in which a call on `device` allocates and launches; gives the stream handle."""
    if stream is None and _torch.cuda.current_device() == device.index:
        return _Current(_raw_stream(device.index))
    return _on(device, stream)


def packer(args):
    """A function that makes the bytes of an argument structure from all of its fields, in
    order (pointers as integers): filling the ctypes structure itself takes three times as
    long, and a call of few tokens takes as long as its host side."""
    codes = {ctypes.c_void_p: "P", ctypes.c_size_t: "N", ctypes.c_int64: "q", ctypes.c_int32: "i"}
    made = struct.Struct("@" + "".join(codes[kind] for _, kind in args._fields_))
    if made.size != ctypes.sizeof(args):
        raise TypeError(f"{args.__name__} ends in padding")
    return made.pack


def new_state(like, state_in, shape, dtype):
    """An uninitialised contiguous state."""
    if state_in is not None:  # checked: contiguous and of that shape and dtype
        return _torch.empty_like(state_in)
    return like.new_empty(shape, dtype=dtype)


def sequences(cu_seqlens, B):
    """The number of sequences of a call: B, or those that cu_seqlens packs into one row."""
    if cu_seqlens is None:
        return B
    is_tensor(cu_seqlens, "cu_seqlens", _torch.int64)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise KdaError(2, "cu_seqlens must be a 1-D tensor of N + 1 >= 2 offsets")
    if not cu_seqlens.is_contiguous():
        raise KdaError(2, "cu_seqlens must be contiguous")
    if B != 1:
        raise KdaError(2, f"packed varlen needs B = 1 (got {B})")
    return cu_seqlens.numel() - 1


def channel_strides(t, name, B, T):
    """Batch and token stride of a [B, T, channels] tensor whose channels are contiguous."""
    s = t.stride()
    if s[2] != 1 and t.shape[2] != 1 and B and T:
        raise KdaError(2, f"the last axis of {name} must be contiguous")
    # the stride of an axis of one entry says nothing
    return (0 if B == 1 else s[0]), (0 if T == 1 else s[1])


def _state_check(t, name, shape, dtype):
    if t.shape != shape:
        raise KdaError(2, f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.dtype != dtype:
        raise KdaError(3, f"{name} is {t.dtype}, the state dtype is {dtype}")


def states(state_in, state_out, state_dtype, io_dtype, N, a, b, ssm_state_indices,
           state_out_indices):
    """Checks of the state arguments of an operator whose states are [N, a, b] (with
    ssm_state_indices a pool [slots, a, b]): (state_out, dtype, its code, slots, pitch)."""
    torch = _torch
    if state_in is not None:
        is_tensor(state_in, "state_in")
    if state_dtype is None:
        state_dtype = io_dtype if state_in is None else state_in.dtype
    code = KDA_FP32 if state_dtype == torch.float32 else KDA_BF16
    if code == KDA_BF16 and state_dtype != torch.bfloat16:
        raise KdaError(3, f"state dtype {state_dtype}")
    if ssm_state_indices is None:
        if state_out_indices is not None:
            raise KdaError(10, "state_out_indices needs ssm_state_indices")
        shape = (N, a, b)
        if state_in is not None:
            _state_check(state_in, "state_in", shape, state_dtype)
            if not state_in.is_contiguous():
                raise KdaError(2, "state_in must be contiguous")
        if state_out is not None and state_out is not state_in:
            is_tensor(state_out, "state_out")
            _state_check(state_out, "state_out", shape, state_dtype)
            if not state_out.is_contiguous():
                raise KdaError(2, "state_out must be contiguous")
        return state_out, state_dtype, code, 0, 0
    if state_in is None:
        raise KdaError(10, "a state pool needs state_in")
    if state_in.dim() != 3 or state_in.shape[0] < 1:
        raise KdaError(2, f"a state pool needs state_in [slots, {a}, {b}]")
    slots = state_in.shape[0]
    _state_check(state_in, "the state pool", (slots, a, b), state_dtype)
    st = state_in.stride()
    if st[2] != 1 or (a > 1 and st[1] != b):
        raise KdaError(2, "each state pool slot must be contiguous")
    pitch = st[0] if slots > 1 else a * b
    if pitch < a * b:  # 0 would be taken for dense slots
        raise KdaError(10, f"the state pool's slot pitch {pitch} is less than a slot")
    if pitch % 8:
        raise KdaError(2, "the state pool's slot pitch must be a multiple of 8 elements")
    if state_out is not None and state_out is not state_in:
        is_tensor(state_out, "state_out")
        if state_out.data_ptr() != state_in.data_ptr():
            raise KdaError(6, "with a state pool, state_out must be None or state_in")
    for name, ids in (("ssm_state_indices", ssm_state_indices),
                      ("state_out_indices", state_out_indices)):
        if ids is not None:
            is_tensor(ids, name, torch.int32)
            if ids.shape != (N,) or not ids.is_contiguous():
                raise KdaError(2, f"{name} must be a contiguous [{N}]")
    return state_in, state_dtype, code, slots, pitch


def vector(t, name, n):
    """An optional FP32 [n]."""
    if t is not None:
        is_tensor(t, name, _torch.float32)
        if t.shape != (n,) or not t.is_contiguous():
            raise KdaError(2, f"{name} must be a contiguous [{n}]")
