"""What the bindings of the operators beside kda_prefill share: checks of tensors, and the
stream and device a call runs on. These calls can take a few microseconds on the device, so
the checks of the common case are kept short."""

import contextlib

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
    for i, t in enumerate((first, *rest)):
        if t is not None and (index < 0 or t.get_device() != index):
            raise KdaError(2, f"{names.split()[i]} must be a CUDA tensor on "
                           f"{first.device if index >= 0 else 'cuda'} (got {t.device})")
    return first.device


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
