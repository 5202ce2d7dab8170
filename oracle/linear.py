"""FP64 oracle of linear attention with one decay per head, the state pool's slot operations
and the gated norm: the definitions, one token, slot or row after another. Test
infrastructure only; shares no code with the HIP path.
"""

import numpy as np


def linear_recurrence_fp64(q, k, v, g=None, state0=None, *, log_decay=None, cu_seqlens=None,
                           scale=None):
    """q, k [B, T, Hk, K], v [B, T, H, V], g [B, T, H]: (o, state, o_abs, state_abs). The last
    two are the same sums over the terms' absolute values: what a rounding of every term by
    at most r can move the results by is at most r times them."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, T, Hk, K = q.shape
    H, V = v.shape[2:]
    scale = K ** -0.5 if scale is None else scale
    ld = np.zeros((B, T, H)) if g is None else np.asarray(g, np.float64).copy()
    if log_decay is not None:
        ld = ld + np.asarray(log_decay, np.float64)
    if cu_seqlens is None:
        spans = [(b, 0, T) for b in range(B)]
    else:
        cu = [int(x) for x in cu_seqlens]
        spans = [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]
    rep = H // Hk
    o = np.zeros((B, T, H, V))
    o_abs = np.zeros_like(o)
    state = np.zeros((len(spans), H, V, K))
    state_abs = np.zeros_like(state)
    for n, (b, lo, hi) in enumerate(spans):
        S = np.zeros((H, V, K)) if state0 is None else np.array(state0[n], np.float64)
        A = np.abs(S)
        for t in range(lo, hi):
            kt, qt = np.repeat(k[b, t], rep, 0), np.repeat(q[b, t], rep, 0)
            d = np.exp(ld[b, t])[:, None, None]
            w = v[b, t][:, :, None] * kt[:, None, :]
            S = d * S + w
            A = d * A + np.abs(w)
            o[b, t] = scale * np.einsum("hvk,hk->hv", S, qt)
            o_abs[b, t] = scale * np.einsum("hvk,hk->hv", A, np.abs(qt))
        state[n], state_abs[n] = S, A
    return o, state, o_abs, state_abs


def compact_slots(ids, slots):
    """(new ids, live count, moves) of the compaction of `ids` in a pool of `slots`."""
    live = sorted({int(i) for i in ids if 0 <= i < slots})
    count = len(live)
    held = set(live)
    holes = [s for s in range(count) if s not in held]
    moves = dict(zip([s for s in live if s >= count], holes))
    return [moves.get(int(i), int(i)) for i in ids], count, moves


def gated_norm_fp64(x, gate=None, weight=None, residual=None, *, next_weight=None, eps=1e-6,
                    act="sigmoid", scale=1.0, next_norm=False):
    x = np.asarray(x, np.float64)
    y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if gate is not None:
        e = np.asarray(gate, np.float64)
        s = 1 / (1 + np.exp(-e))
        y = y * (e * s if act == "silu" else s)
    y = y * scale
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    if next_weight is None and not next_norm:
        return y
    z = y / np.sqrt(np.mean(y * y, -1, keepdims=True) + eps)
    return y, z if next_weight is None else z * np.asarray(next_weight, np.float64)
