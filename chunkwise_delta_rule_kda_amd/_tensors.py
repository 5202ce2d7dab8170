"""What the bindings of the operators beside kda_prefill share: checks of tensors, and the
stream and device a call runs on."""

import contextlib

from . import KDA_BF16, KDA_FP32, KdaError


def need(cond, status, msg):
    if not cond:
        raise KdaError(status, msg)


def dtype_code(t, name):
    import torch

    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_FP32
    raise KdaError(3, f"{name} has unsupported dtype {t.dtype}")


def is_tensor(t, name, dtype=None):
    import torch

    need(isinstance(t, torch.Tensor), 2, f"{name} must be a tensor")
    need(dtype is None or t.dtype == dtype, 3, f"{name} is {t.dtype}, expected {dtype}")


def on_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and (not t.is_cuda or t.device != device):
            raise KdaError(2, f"{name} must be a CUDA tensor on {device} (got {t.device})")


def steps(t):
    """Strides in elements, 0 for axes of one entry (their stride says nothing)."""
    return [s if n != 1 else 0 for s, n in zip(t.stride(), t.shape)]


@contextlib.contextmanager
def _on(device, stream):
    import torch

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
    import torch

    if stream is None and torch.cuda.current_device() == device.index:
        return _Current(torch.cuda.current_stream(device).cuda_stream)
    return _on(device, stream)
