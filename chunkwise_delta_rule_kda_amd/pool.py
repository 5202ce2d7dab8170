"""Slots of a state pool: bindings of kda_pool_copy and kda_pool_compact (include/kda.h)."""

import ctypes

from . import KdaError, kda_last_error, load_library
from ._tensors import dtype_code, get_torch, is_tensor, need, on_device, run_on

__all__ = ["kda_pool", "kda_pool_copy", "kda_pool_copy_args", "kda_pool_compact",
           "kda_pool_compact_args", "KDA_POOL_COMPACT_SLOTS"]

KDA_POOL_COMPACT_SLOTS = 1 << 18  # include/kda.h

_P, _I64 = ctypes.c_void_p, ctypes.c_int64


class kda_pool(ctypes.Structure):
    _fields_ = [("base", _P), ("slots", _I64), ("layers", _I64), ("slot_elems", _I64),
                ("slot_pitch", _I64), ("layer_pitch", _I64), ("dtype", ctypes.c_int32)]


class kda_pool_copy_args(ctypes.Structure):
    _fields_ = [("src", kda_pool), ("dst", kda_pool), ("src_idx", _P), ("dst_idx", _P),
                ("pairs", _I64)]


class kda_pool_compact_args(ctypes.Structure):
    _fields_ = [("pool", kda_pool), ("idx", _P), ("new_idx", _P), ("count", _P), ("n", _I64),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


def _pool_of(t, name, layered):
    """[slots, ...] (or [layers, slots, ...]) with contiguous slots, as a kda_pool."""
    get_torch()
    is_tensor(t, name)
    code = dtype_code(t, name)
    axis = 1 if layered else 0
    if not (t.dim() >= axis + 2):
        raise KdaError(2, f"{name} must be [{'layers, ' if layered else ''}slots, ...]")
    shape, stride = t.shape, t.stride()
    elems = 1
    for n, s in zip(reversed(shape[axis + 1:]), reversed(stride[axis + 1:])):
        if not (n == 1 or s == elems):
            raise KdaError(2, f"each slot of {name} must be contiguous")
        elems *= n
    if not (elems >= 1 and shape[axis] >= 1 and (not layered or shape[0] >= 1)):
        raise KdaError(2, f"{name} is empty")
    pitch = stride[axis] if shape[axis] > 1 else elems
    layers = shape[0] if layered else 1
    return kda_pool(t.data_ptr(), shape[axis], layers, elems, pitch,
                    stride[0] if layers > 1 else 0, code)


def _index(t, name):
    is_tensor(t, name, get_torch().int32)
    if not (t.dim() == 1 and t.is_contiguous()):
        raise KdaError(2, f"{name} must be a contiguous 1-D tensor")


def kda_pool_copy(pool, src, dst, *, source=None, layered=False, stream=None):
    """pool[dst[i]] <- source[src[i]] for every i, in one launch: copies of slots, forks
    (one source in several pairs), restores from another pool or a checkpoint buffer (also
    between bf16 and fp32), and clears (a src id outside the source writes zeros).

    pool: [slots, ...], e.g. [slots, H, 128, 128]; source: the same but for its number of
    slots, or None (the pool itself). layered: both start with an axis of layers, and a
    pair names the slot in all of them. Slots have to be contiguous, the axes of slots and
    layers may be padded. src, dst: int32 [pairs]. A dst id outside the pool writes
    nothing. Destinations must be distinct and no other pair's source (caller contract,
    not checked). Returns pool.
    """
    d = _pool_of(pool, "pool", layered)
    s = d if source is None or source is pool else _pool_of(source, "source", layered)
    need(s.slot_elems == d.slot_elems and s.layers == d.layers, 2,
         "pool and source differ in their layers or slots")
    _index(src, "src")
    _index(dst, "dst")
    if not (src.numel() == dst.numel()):
        raise KdaError(2, f"src has {src.numel()} ids, dst {dst.numel()}")
    dev = on_device(pool, "pool source src dst", source, src, dst)
    a = kda_pool_copy_args(s, d, src.data_ptr(), dst.data_ptr(), src.numel())
    with run_on(dev, stream) as handle:
        status = load_library().kda_pool_copy(ctypes.byref(a), handle)
    if status:
        raise KdaError(status, kda_last_error())
    return pool


def kda_pool_compact(pool, slots, *, new_slots=None, count=None, workspace=None, layered=False,
                     stream=None):
    """Move as few slots as possible so that the live ones are the pool's first ones.

    pool: as in kda_pool_copy. slots: int32 [n], the slots in use (ids outside the pool are
    handed through; an id may appear more than once). With L distinct live slots, the k-th
    live slot >= L is copied to the k-th free slot < L; the others stay. Returns (new_slots
    int32 [n], count int32 [1]): the slot each entry of `slots` has afterwards, and L.
    new_slots may be `slots` itself. Everything happens on the device: nothing is read
    back to the host. A pool has at most KDA_POOL_COMPACT_SLOTS slots here.
    """
    torch = get_torch()
    p = _pool_of(pool, "pool", layered)
    _index(slots, "slots")
    n = slots.numel()
    if new_slots is not None:
        _index(new_slots, "new_slots")
        if not (new_slots.numel() == n):
            raise KdaError(2, f"new_slots must have {n} entries")
    if count is not None:
        _index(count, "count")
        need(count.numel() == 1, 2, "count must have one entry")
    if workspace is not None:
        is_tensor(workspace, "workspace")
        need(workspace.is_contiguous(), 2, "workspace must be contiguous")
    dev = on_device(pool, "pool slots new_slots count workspace", slots, new_slots, count,
                    workspace)
    lib = load_library()
    with run_on(dev, stream) as handle:
        if new_slots is None:
            new_slots = torch.empty_like(slots)
        if count is None:
            count = slots.new_empty(1)
        a = kda_pool_compact_args(p, slots.data_ptr(), new_slots.data_ptr(), count.data_ptr(), n,
                                  None, 0)
        if workspace is None:
            size = ctypes.c_size_t(0)
            status = lib.kda_pool_compact_workspace_bytes(ctypes.byref(a), ctypes.byref(size))
            if status:
                raise KdaError(status, kda_last_error())
            workspace = slots.new_empty(size.value // 4)  # a multiple of 256 bytes
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
        status = lib.kda_pool_compact(ctypes.byref(a), handle)
    if status:
        raise KdaError(status, kda_last_error())
    return new_slots, count
