"""FP64 oracle of the short causal convolution and the selective state space scan: the
definitions, one token after another, with bounds on what FP32 arithmetic may be off. Test
infrastructure only; shares no code with the HIP path.
"""

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, np.float64)


def _spans(B, T, cu_seqlens):
    if cu_seqlens is None:
        return [(b, 0, T) for b in range(B)]
    cu = [int(x) for x in cu_seqlens]
    return [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]


def _silu(x):
    with np.errstate(over="ignore"):
        return x / (1 + np.exp(-x))


def _silu_error(x):
    """Of silu in FP32, in units of 2^-24 |silu(x)|: the exponent's rounding (|x|), the
    exponential, the sum, the reciprocal and the product."""
    return np.abs(x) + 8


def short_conv_fp64(x, weight, bias=None, state0=None, *, cu_seqlens=None, silu=True):
    """x [B, T, C], weight [C, W], state0 [N, W-1, C]: (y, state, error), the error in units
    of 2^-24: W products and sums of the taps, and the activation's (its slope is at most
    1.1)."""
    x, weight, bias, state0 = _f64(x), _f64(weight), _f64(bias), _f64(state0)
    B, T, C = x.shape
    W = weight.shape[1]
    spans = _spans(B, T, cu_seqlens)
    y, err = np.zeros_like(x), np.zeros_like(x)
    state = np.zeros((len(spans), W - 1, C))
    for n, (b, lo, hi) in enumerate(spans):
        rows = list(np.zeros((W - 1, C)) if state0 is None else state0[n])
        for t in range(lo, hi):
            rows.append(x[b, t])
            taps = [weight[:, i] * rows[-W + i] for i in range(W)]
            a = sum(taps) + (0 if bias is None else bias)
            e = (W + 1) * (sum(np.abs(v) for v in taps) + (0 if bias is None else np.abs(bias)))
            y[b, t] = _silu(a) if silu else a
            err[b, t] = 1.1 * e + _silu_error(a) * np.abs(y[b, t]) if silu else e
        state[n] = rows[len(rows) - (W - 1):]
    return y, state, err


def selective_scan_fp64(u, delta, A, B, C, D=None, z=None, state0=None, *, delta_bias=None,
                        softplus=True, cu_seqlens=None, segment=0):
    """u, delta, z [B, T, D], A [D, S], B, C [B, T, G, S], state0 [N, D, S]:
    (y, state, y_error, state_error), the errors in units of 2^-24: bounds on what FP32
    arithmetic is off, carried along with the recurrence.

    The step size d is off by (14 + 3 |x|) units of its own (x the softplus' argument; the
    exponent and the argument's sum give the |x|; exponential, reciprocal, polynomial and
    products the rest), or by 1 as it is. A decay exp(d A) then is off by |d A| (that + 3) + 2
    (A times log2 e, their product, the exponential), where a segment's end state is carried
    over `segment` tokens by their sum of step sizes, by |d A| segment more; the written term
    by that + 2; and the new state is rounded once.
    """
    u, delta, A, B, C, D, z, state0, delta_bias = (
        _f64(x) for x in (u, delta, A, B, C, D, z, state0, delta_bias))
    Bt, T, ch = u.shape
    G, S = B.shape[2:]
    spans = _spans(Bt, T, cu_seqlens)
    y, y_err = np.zeros_like(u), np.zeros_like(u)
    state, state_err = np.zeros((len(spans), ch, S)), np.zeros((len(spans), ch, S))
    for n, (b, lo, hi) in enumerate(spans):
        h = np.zeros((ch, S)) if state0 is None else state0[n].copy()
        top, err = np.abs(h), np.zeros((ch, S))  # sum of absolute terms, error
        for t in range(lo, hi):
            x = delta[b, t] + (0 if delta_bias is None else delta_bias)
            d = np.logaddexp(x, 0) if softplus else x
            off = ((14 + 3 * np.abs(x)) if softplus else np.ones(ch))[:, None]
            arg = d[:, None] * A
            a = np.exp(arg)
            Bn, Cn = (np.repeat(m[b, t], ch // G, 0) for m in (B, C))
            w = (d * u[b, t])[:, None] * Bn
            err = a * (err + top * (np.abs(arg) * (off + 3 + segment) + 2)) + np.abs(w) * (off + 2)
            h = a * h + w
            top = a * top + np.abs(w)
            err = err + top
            o = (h * Cn).sum(-1)
            o_top = (top * np.abs(Cn)).sum(-1)
            e = (err * np.abs(Cn)).sum(-1) + (S + 4) * o_top
            if D is not None:
                o = o + D * u[b, t]
                e = e + 2 * (o_top + np.abs(D * u[b, t]))
            if z is not None:
                s = _silu(z[b, t])
                e = e * np.abs(s) + np.abs(o * s) * (_silu_error(z[b, t]) + 1)
                o = o * s
            y[b, t], y_err[b, t] = o, e
        state[n], state_err[n] = h, err
    return y, state, y_err, state_err
