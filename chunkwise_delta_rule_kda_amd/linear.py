"""Linear attention with one decay per head: binding of kda_linear (include/kda.h)."""

import ctypes

from . import KdaError, _raise_if, kda_last_error, load_library
from ._tensors import contiguous_like, dtype_code, get_torch, is_tensor, need, on_device, run_on

__all__ = ["kda_linear", "kda_linear_args", "kda_linear_check", "kda_linear_plan",
           "kda_linear_workspace_bytes", "make_linear_args"]

_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class kda_linear_args(ctypes.Structure):
    _fields_ = (
        [(n, _P) for n in ("q", "k", "v", "g", "log_decay", "state_in", "cu_seqlens", "o",
                           "state_out", "workspace")]
        + [("workspace_bytes", ctypes.c_size_t)]
        + [(n, _I64) for n in ("B", "T", "H", "Hk", "K", "V", "N")]
        + [(f"{x}_stride_{d}", _I64) for x in "qkv" for d in ("batch", "token", "head")]
        + [(n, _I32) for n in ("io_dtype", "state_dtype", "g_dtype")]
        + [("scale", ctypes.c_float), ("segment_tokens", _I64), ("ssm_state_indices", _P),
           ("state_out_indices", _P), ("state_pool_slots", _I64), ("state_slot_pitch", _I64)])


class kda_linear_plan_info(ctypes.Structure):
    _fields_ = [("decode", _I32), ("value_block", _I32), ("segment_tokens", _I64),
                ("segments_bound", _I64), ("workgroups", _I64), ("state_workgroups", _I64),
                ("workspace_bytes", ctypes.c_size_t)]


def _ptr(x):
    return x if x is None or isinstance(x, int) else x.data_ptr()


def make_linear_args(*, B, T, H, N, Hk=None, K=128, V=128, io_dtype=0, state_dtype=0,
                     g_dtype=1, q_stride=None, k_stride=None, v_stride=None, **kw):
    """Fill a kda_linear_args from raw pointers (ints), tensors or None; strides default to
    contiguous tensors."""
    Hk = H if Hk is None else Hk
    a = kda_linear_args()
    a.B, a.T, a.H, a.Hk, a.K, a.V, a.N = B, T, H, Hk, K, V, N
    a.io_dtype, a.state_dtype, a.g_dtype = io_dtype, state_dtype, g_dtype
    for x, st, heads, dim in (("q", q_stride, Hk, K), ("k", k_stride, Hk, K),
                              ("v", v_stride, H, V)):
        for d, s in zip(("batch", "token", "head"), st or (T * heads * dim, heads * dim, dim)):
            setattr(a, f"{x}_stride_{d}", s)
    for name, x in kw.items():
        if name in ("scale", "segment_tokens", "workspace_bytes", "state_pool_slots",
                    "state_slot_pitch"):
            setattr(a, name, x)
        else:
            setattr(a, name, _ptr(x))
    return a


def kda_linear_workspace_bytes(args):
    n = ctypes.c_size_t(0)
    _raise_if(load_library().kda_linear_workspace_bytes(ctypes.byref(args), ctypes.byref(n)))
    return n.value


def kda_linear_check(args):
    """Host-only validation; returns the status code (0 = OK)."""
    return load_library().kda_linear_check(ctypes.byref(args))


def kda_linear_plan(args):
    info = kda_linear_plan_info()
    _raise_if(load_library().kda_linear_plan(ctypes.byref(args), ctypes.byref(info)))
    return {f: getattr(info, f) for f, _ in kda_linear_plan_info._fields_}


def _state_check(t, name, shape, dtype):
    if t.shape != shape:
        raise KdaError(2, f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.dtype != dtype:
        raise KdaError(3, f"{name} is {t.dtype}, the state dtype is {dtype}")


def kda_linear(q, k, v, g=None, state_in=None, cu_seqlens=None, *, log_decay=None, scale=None,
               output_final_state=True, state_dtype=None, o=None, state_out=None,
               workspace=None, segment_tokens=0, ssm_state_indices=None,
               state_out_indices=None, stream=None):
    """Linear attention with one decay per head, forward, on the current (or given) stream:

        S <- exp(g_t + log_decay) S + v_t k_t^T ;  o_t = scale * S q_t

    q, k: [B, T, Hk, K] (K 64 or 128), v: [B, T, H, V] (V a multiple of 64 up to 512), bf16
    or fp32 CUDA tensors; Hk divides H and head h reads q/k head h // (H // Hk). Only their
    last axis has to be contiguous (the other strides multiples of 8), so slices of one
    projection are taken as they are. g: [B, T, H] log decays (<= 0; -inf empties the
    state) of q's dtype or fp32, or None. log_decay: fp32 [H], a fixed decay of each head,
    or None; where both are given they add. scale: None (or 0) is 1 / sqrt(K).
    state_in: [N, H, V, K] or None (zeros); state_out=state_in updates in place.
    cu_seqlens: int64 [N + 1] (B = 1) or None.
    1 <= T <= 8 in the fixed layout is the step of single (or a few draft) tokens: each state
    is read and written once. segment_tokens: 0 automatic, negative serial, positive the
    time-segment length (a multiple of 64).
    ssm_state_indices (int32 [N]): state_in is a pool [slots, H, V, K] (its first axis may
    be padded), sequence n starts from slot ssm_state_indices[n] and writes its final state
    to slot state_out_indices[n] (None: the slot it read); the returned state is the pool.
    Ids outside the pool start from zero and write nothing.
    Returns (o, state_out or None).
    """
    torch = get_torch()
    is_tensor(q, "q")
    is_tensor(k, "k")
    is_tensor(v, "v")
    if q.dim() != 4 or v.dim() != 4:
        raise KdaError(2, "q and v must have four axes, [B, T, heads, dim]")
    shape = q.shape
    B, T, Hk, K = shape
    vB, vT, H, V = v.shape
    io = dtype_code(q, "q")
    dt = q.dtype
    if k.shape != shape:
        raise KdaError(2, f"k has shape {tuple(k.shape)}, expected {tuple(shape)}")
    if vB != B or vT != T:
        raise KdaError(2, f"v has shape {tuple(v.shape)}, expected ({B}, {T}, heads, dim)")
    if k.dtype != dt or v.dtype != dt:
        raise KdaError(3, f"q, k, v are {dt}, {k.dtype}, {v.dtype}")
    if Hk < 1 or H < 1 or H % Hk:
        raise KdaError(2, f"{Hk} q/k heads do not divide {H} heads")
    sq, sk, sv = q.stride(), k.stride(), v.stride()
    if (sq[3] != 1 or sk[3] != 1 or sv[3] != 1) and B and T:
        raise KdaError(2, "the last axis of q, k and v must be contiguous")
    if B == 1 or T == 1 or Hk == 1 or H == 1:  # the stride of an axis of one entry says nothing
        one = [n == 1 for n in (B, T, Hk, H)]
        sq, sk = ([0 if o else x for o, x in zip(one[:3], st)] for st in (sq, sk))
        sv = [0 if o else x for o, x in zip((one[0], one[1], one[3]), sv)]
    N = B
    if cu_seqlens is not None:
        is_tensor(cu_seqlens, "cu_seqlens", torch.int64)
        need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2, 2,
             "cu_seqlens must be a 1-D tensor of N + 1 >= 2 offsets")
        need(cu_seqlens.is_contiguous(), 2, "cu_seqlens must be contiguous")
        if not (B == 1):
            raise KdaError(2, f"packed varlen needs B = 1 (got {B})")
        N = cu_seqlens.numel() - 1
    gt = 1
    if g is not None:
        is_tensor(g, "g")
        gt = dtype_code(g, "g")
        if gt != 1 and gt != io:
            raise KdaError(3, f"g is {g.dtype}, expected {dt} or float32")
        if g.shape != (B, T, H):
            raise KdaError(2, f"g has shape {tuple(g.shape)}, expected {(B, T, H)}")
        if not g.is_contiguous():
            raise KdaError(2, "g must be contiguous")
    if log_decay is not None:
        is_tensor(log_decay, "log_decay", torch.float32)
        if not (log_decay.shape == (H,) and log_decay.is_contiguous()):
            raise KdaError(2, f"log_decay must be a contiguous [{H}]")
    if state_in is not None:
        is_tensor(state_in, "state_in")
    if state_dtype is None:
        state_dtype = state_in.dtype if state_in is not None else dt
    st_code = 0 if state_dtype == torch.bfloat16 else 1
    if st_code and state_dtype != torch.float32:
        raise KdaError(3, f"state dtype {state_dtype}")
    slots = pitch = 0
    if ssm_state_indices is not None:
        need(state_in is not None, 10, "a state pool needs state_in")
        need(state_in.dim() == 4 and state_in.shape[0] >= 1, 2,
             "a state pool needs state_in [slots, H, V, K]")
        slots = state_in.shape[0]
        _state_check(state_in, "the state pool", (slots, H, V, K), state_dtype)
        st = state_in.stride()
        if st[3] != 1 or st[2] != K or (H > 1 and st[1] != V * K):
            raise KdaError(2, "each state pool slot must be contiguous")
        pitch = st[0] if slots > 1 else H * V * K
        if pitch < H * V * K:  # 0 would be taken for dense slots
            raise KdaError(10, f"the state pool's slot pitch {pitch} is less than a slot")
        if pitch % 8:
            raise KdaError(2, "the state pool's slot pitch must be a multiple of 8 elements")
        if state_out is not None and state_out is not state_in:
            is_tensor(state_out, "state_out")
            if state_out.data_ptr() != state_in.data_ptr():
                raise KdaError(6, "with a state pool, state_out must be None or state_in")
        state_out = state_in
        for name, ids in (("ssm_state_indices", ssm_state_indices),
                          ("state_out_indices", state_out_indices)):
            if ids is not None:
                is_tensor(ids, name, torch.int32)
                if ids.shape != (N,) or not ids.is_contiguous():
                    raise KdaError(2, f"{name} must be a contiguous [{N}]")
    else:
        need(state_out_indices is None, 10, "state_out_indices needs ssm_state_indices")
        for name, t in (("state_in", state_in), ("state_out", state_out)):
            if t is not None:
                is_tensor(t, name)
                _state_check(t, name, (N, H, V, K), state_dtype)
                if not t.is_contiguous():
                    raise KdaError(2, f"{name} must be contiguous")
    if o is not None:
        is_tensor(o, "o")
        if not (o.shape == v.shape and o.dtype == dt and o.is_contiguous()):
            raise KdaError(2, f"o must be a contiguous {tuple(v.shape)} of {dt}")
    if workspace is not None:
        is_tensor(workspace, "workspace")
        need(workspace.is_contiguous(), 2, "workspace must be contiguous")
    dev = on_device(q, "q k v g log_decay state_in cu_seqlens o state_out workspace "
                    "ssm_state_indices state_out_indices", k, v, g, log_decay, state_in, cu_seqlens,
                    o, state_out, workspace, ssm_state_indices, state_out_indices)
    lib = load_library()
    with run_on(dev, stream) as handle:
        if o is None:
            o = contiguous_like(v)
        if state_out is None and output_final_state:
            state_out = (torch.empty_like(state_in) if state_in is not None
                         else v.new_empty((N, H, V, K), dtype=state_dtype))
        a = kda_linear_args(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(g), _ptr(log_decay), _ptr(state_in),
            _ptr(cu_seqlens), o.data_ptr(), _ptr(state_out), None, 0, B, T, H, Hk, K, V, N,
            sq[0], sq[1], sq[2], sk[0], sk[1], sk[2], sv[0], sv[1], sv[2], io, st_code, gt,
            0.0 if scale is None else scale, segment_tokens, _ptr(ssm_state_indices),
            _ptr(state_out_indices), slots, pitch)
        ref = ctypes.byref(a)
        if workspace is not None:
            a.workspace = workspace.data_ptr()
            a.workspace_bytes = workspace.numel() * workspace.element_size()
        status = lib.kda_linear(ref, handle)
        if status == 7 and workspace is None:  # the call needs one: refused before any launch
            workspace = torch.empty(kda_linear_workspace_bytes(a), dtype=torch.uint8, device=dev)
            a.workspace = workspace.data_ptr()
            a.workspace_bytes = workspace.numel()
            status = lib.kda_linear(ref, handle)
    if status:
        raise KdaError(status, kda_last_error())
    return o, state_out
