"""The selective state space scan: binding of kda_selective_scan (include/kda.h)."""

import ctypes

from . import KdaError, _raise_if, kda_last_error, load_library
from ._tensors import (channel_strides, contiguous_like, dtype_code, get_torch, is_tensor, need,
                       new_state, on_device, packer, run_on, sequences, states, vector)

__all__ = ["kda_selective_scan", "kda_selective_scan_args", "kda_selective_scan_check",
           "kda_selective_scan_plan", "kda_selective_scan_workspace_bytes",
           "make_selective_scan_args"]

_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32

_SOFTPLUS = 1  # KDA_SCAN_SOFTPLUS


class kda_selective_scan_args(ctypes.Structure):
    _fields_ = (
        [(n, _P) for n in ("u", "delta", "z", "B_in", "C_in", "A", "D_skip", "delta_bias",
                           "state_in", "cu_seqlens", "out", "state_out", "workspace")]
        + [("workspace_bytes", ctypes.c_size_t)]
        + [(n, _I64) for n in ("B", "T", "D", "S", "G", "N")]
        + [(f"{x}_stride_{d}", _I64) for x in ("u", "delta", "z") for d in ("batch", "token")]
        + [(f"{x}_stride_{d}", _I64) for x in "BC" for d in ("batch", "token", "group")]
        + [(n, _I32) for n in ("io_dtype", "state_dtype", "flags")]
        + [("segment_tokens", _I64), ("ssm_state_indices", _P), ("state_out_indices", _P),
           ("state_pool_slots", _I64), ("state_slot_pitch", _I64)])


_pack = packer(kda_selective_scan_args)


class kda_selective_scan_plan_info(ctypes.Structure):
    _fields_ = [("decode", _I32), ("segment_tokens", _I64), ("segments_bound", _I64),
                ("workgroups", _I64), ("workspace_bytes", ctypes.c_size_t)]


def _ptr(x):
    return x if x is None or isinstance(x, int) else x.data_ptr()


def make_selective_scan_args(*, B, T, D, N, S=16, G=1, u_stride=None, delta_stride=None,
                             z_stride=None, B_stride=None, C_stride=None, **kw):
    """Fill a kda_selective_scan_args from raw pointers (ints), tensors or None; strides
    default to contiguous tensors."""
    a = kda_selective_scan_args()
    a.B, a.T, a.D, a.S, a.G, a.N = B, T, D, S, G, N
    for x, st in (("u", u_stride), ("delta", delta_stride), ("z", z_stride)):
        for d, s in zip(("batch", "token"), st or (T * D, D)):
            setattr(a, f"{x}_stride_{d}", s)
    for x, st in (("B", B_stride), ("C", C_stride)):
        for d, s in zip(("batch", "token", "group"), st or (T * G * S, G * S, S)):
            setattr(a, f"{x}_stride_{d}", s)
    for name, x in kw.items():
        whole = name in ("io_dtype", "state_dtype", "flags", "segment_tokens", "workspace_bytes",
                         "state_pool_slots", "state_slot_pitch")
        setattr(a, name, x if whole else _ptr(x))
    return a


def kda_selective_scan_workspace_bytes(args):
    n = ctypes.c_size_t(0)
    _raise_if(load_library().kda_selective_scan_workspace_bytes(ctypes.byref(args),
                                                                ctypes.byref(n)))
    return n.value


def kda_selective_scan_check(args):
    """Host-only validation; returns the status code (0 = OK)."""
    return load_library().kda_selective_scan_check(ctypes.byref(args))


def kda_selective_scan_plan(args):
    info = kda_selective_scan_plan_info()
    _raise_if(load_library().kda_selective_scan_plan(ctypes.byref(args), ctypes.byref(info)))
    return {f: getattr(info, f) for f, _ in kda_selective_scan_plan_info._fields_}


def kda_selective_scan(u, delta, A, B, C, D=None, z=None, state_in=None, cu_seqlens=None, *,
                       delta_bias=None, delta_softplus=True, output_final_state=True,
                       state_dtype=None, out=None, state_out=None, workspace=None,
                       segment_tokens=0, ssm_state_indices=None, state_out_indices=None,
                       stream=None):
    """Selective state space scan, forward, on the current (or given) stream. For every
    channel c and its S states:

        d = softplus(delta_t + delta_bias)
        h <- exp(d A) h + d u_t B_t ;  out_t = (C_t . h + D u_t) z_t sigmoid(z_t)

    in fp32, out rounded once. u, delta, z: [B, T, channels], bf16 or fp32, channels a
    multiple of 8 (z None: no gate). A: fp32 [channels, S], finite and negative; S 8, 16, 32
    or 64. B, C: [B, T, S], or [B, T, G, S] where channel c reads group c // (channels // G)
    (groups of a multiple of 32 channels). D, delta_bias: fp32 [channels] or None.
    delta_softplus=False takes delta + delta_bias as the step size. Of u, delta, z, B and C
    only the last axis has to be contiguous (the other strides multiples of 8, the tokens' at
    most 2^22), so slices of projections are taken as they are. Tensors other than D and
    delta_bias start on multiples of 16 bytes.
    state_in: [N, channels, S] or None (zeros); state_out=state_in updates in place.
    state_dtype: the states' type, bf16 or fp32; None is state_in's, or without one u's. With
    bf16 inputs ask for torch.float32 where the state is carried from call to call: a bf16 one
    is rounded in each, and under a decay closer to 1 than 2^-9 it does not move at all.
    cu_seqlens: int64 [N + 1] (B = 1) or None. 1 <= T <= 8 in the fixed layout is the step of
    single (or a few draft) tokens: each state is read and written once. segment_tokens: 0
    automatic, negative serial, positive the time-segment length (a multiple of 64). Packed
    lengths are known on the device only, and the automatic rule takes the longest for 1.75
    times the mean: where one prompt is packed with many short sequences, pass a length
    (1536 channels, 8000 tokens and 63 single ones: 119 us with 512, 312 without).
    ssm_state_indices (int32 [N]): state_in is a pool [slots, channels, S] (its first axis may
    be padded), sequence n starts from slot ssm_state_indices[n] and writes its final state
    to slot state_out_indices[n] (None: the slot it read); the returned state is the pool.
    Ids outside the pool start from zero and write nothing.
    Returns (out, state_out or None).
    """
    torch = get_torch()
    is_tensor(u, "u")
    if u.dim() != 3:
        raise KdaError(2, "u must have three axes, [B, T, channels]")
    shape = u.shape
    batch, T, channels = shape
    io, dt = dtype_code(u, "u"), u.dtype
    is_tensor(delta, "delta", dt)
    if delta.shape != shape:
        raise KdaError(2, f"delta has shape {tuple(delta.shape)}, expected {tuple(shape)}")
    ub, ut = channel_strides(u, "u", batch, T)
    db, dt_ = channel_strides(delta, "delta", batch, T)
    zb = zt = 0
    if z is not None:
        is_tensor(z, "z", dt)
        if z.shape != shape:
            raise KdaError(2, f"z has shape {tuple(z.shape)}, expected {tuple(shape)}")
        zb, zt = channel_strides(z, "z", batch, T)
    is_tensor(A, "A", torch.float32)
    if A.dim() != 2 or A.shape[0] != channels or not A.is_contiguous():
        raise KdaError(2, f"A must be a contiguous [{channels}, states]")
    S = A.shape[1]
    is_tensor(B, "B", dt)
    is_tensor(C, "C", dt)
    grouped = B.dim() == 4
    G = B.shape[2] if grouped else 1
    rows = (batch, T, G, S) if grouped else (batch, T, S)
    if B.shape != rows or C.shape != rows:
        raise KdaError(2, f"B and C have shapes {tuple(B.shape)} and {tuple(C.shape)}, "
                       f"expected {rows}")
    sB, sC = B.stride(), C.stride()
    if (sB[-1] != 1 or sC[-1] != 1) and batch and T:
        raise KdaError(2, "the last axis of B and C must be contiguous")
    # the stride of an axis of one entry says nothing
    Bb, Cb = (0, 0) if batch == 1 else (sB[0], sC[0])
    Bt, Ct = (0, 0) if T == 1 else (sB[1], sC[1])
    Bg, Cg = (0, 0) if G == 1 else (sB[2], sC[2])
    if G < 1 or channels % G:
        raise KdaError(2, f"{G} groups do not divide {channels} channels")
    vector(D, "D", channels)
    vector(delta_bias, "delta_bias", channels)
    N = sequences(cu_seqlens, batch)
    state_out, state_dtype, code, slots, pitch = states(
        state_in, state_out, state_dtype, dt, N, channels, S, ssm_state_indices,
        state_out_indices)
    if out is not None:
        is_tensor(out, "out")
        if not (out.shape == shape and out.dtype == dt and out.is_contiguous()):
            raise KdaError(2, f"out must be a contiguous {tuple(shape)} of {dt}")
    if workspace is not None:
        is_tensor(workspace, "workspace")
        need(workspace.is_contiguous(), 2, "workspace must be contiguous")
    dev = on_device(u, "u delta A B C D z state_in cu_seqlens delta_bias out state_out workspace "
                    "ssm_state_indices state_out_indices", delta, A, B, C, D, z, state_in,
                    cu_seqlens, delta_bias, out, state_out, workspace, ssm_state_indices,
                    state_out_indices)
    lib = load_library()
    with run_on(dev, stream) as handle:
        if out is None:
            out = contiguous_like(u)
        if state_out is None and output_final_state:
            state_out = new_state(u, state_in, (N, channels, S), state_dtype)
        a = _pack(
            *[0 if t is None else t.data_ptr() for t in (
                u, delta, z, B, C, A, D, delta_bias, state_in, cu_seqlens, out, state_out,
                workspace)],
            0 if workspace is None else workspace.numel() * workspace.element_size(),
            batch, T, channels, S, G, N, ub, ut, db, dt_, zb, zt, Bb, Bt, Bg, Cb, Ct, Cg, io, code,
            _SOFTPLUS if delta_softplus else 0, segment_tokens,
            0 if ssm_state_indices is None else ssm_state_indices.data_ptr(),
            0 if state_out_indices is None else state_out_indices.data_ptr(), slots, pitch)
        status = lib.kda_selective_scan(a, handle)
        if status == 7 and workspace is None:  # the call needs one: refused before any launch
            a = kda_selective_scan_args.from_buffer_copy(a)
            workspace = torch.empty(kda_selective_scan_workspace_bytes(a), dtype=torch.uint8,
                                    device=dev)
            a.workspace = workspace.data_ptr()
            a.workspace_bytes = workspace.numel()
            status = lib.kda_selective_scan(ctypes.byref(a), handle)
    if status:
        raise KdaError(status, kda_last_error())
    return out, state_out
