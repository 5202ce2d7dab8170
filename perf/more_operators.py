"""Cases of the short causal convolution and the selective state space scan: their inputs,
their plain forms in elementary torch operations, and the calls of this package that compute
the same.

A case is a dict: "op" names the operator, the rest are its sizes and types.
"""

import torch

own = False

BF16, FP32 = "bf16", "fp32"


def _dt(name):
    return {BF16: torch.bfloat16, FP32: torch.float32}[name]


def _size(name):
    return {BF16: 2, FP32: 4}[name]


# ---------------------------------------------------------------- the cases


def _conv(name=None, *, B=1, T=1, C=768, W=4, io=BF16, st=BF16, act=True, bias=False, varlen=0,
          pool=False, state=True, sliced=False):
    """B sequences of T tokens (varlen: that many sequences packed into T tokens)."""
    c = dict(op="conv", B=B, T=T, C=C, W=W, io=io, st=st, act=act, bias=bias, varlen=varlen,
             pool=pool, state=state, sliced=sliced)
    return dict(c, name=name) if name else c


def _scan(name=None, *, B=1, T=1, D=1536, N=16, G=1, io=BF16, st=FP32, z=True, skip=True,
          softplus=True, varlen=0, pool=False, state=True):
    c = dict(op="scan", B=B, T=T, D=D, N=N, G=G, io=io, st=st, z=z, skip=skip,
             softplus=softplus, varlen=varlen, pool=pool, state=state)
    return dict(c, name=name) if name else c


def listed():
    return [
        # q, k and v of one user's next token in a small layer of 6 heads of 128: latency
        _conv("conv token H6", B=1, T=1, C=2304),
        # q, k and v of a serving batch's next tokens, 24 heads, their last inputs in a pool:
        # read from one slot and written to another (the first token after a fork)
        _conv("conv tokens pool H24", B=128, T=1, C=9216, pool=True),
        # a long prompt on few heads (a tensor-parallel shard)
        _conv("conv prompt H6", B=1, T=8192, C=2304),
        # the same prompt on a whole layer of 96 heads
        _conv("conv prompt H96", B=1, T=8192, C=36864),
        # a packed batch of prompts in FP32: one half of each row of a projection, three taps
        _conv("conv packed fp32", T=18001, C=1536, W=3, io=FP32, st=FP32, bias=True, varlen=8,
              sliced=True),
        # one user's next token in a state space layer: latency
        _scan("scan token D1536", B=1, T=1, D=1536),
        # a serving batch's next tokens, FP32 states in a pool, read from one slot and written
        # to another
        _scan("scan tokens pool D8192", B=128, T=1, D=8192, pool=True),
        # draft tokens of 32 sequences to be verified
        _scan("scan draft tokens D4096", B=32, T=5, D=4096),
        # a long prompt in a small layer (or a tensor-parallel shard of a larger one)
        _scan("scan prompt D1536", B=1, T=8192, D=1536),
        # a long prompt in a wide layer
        _scan("scan prompt D8192", B=1, T=8192, D=8192),
        # a packed batch of prompts with initial states
        _scan("scan packed D4096", T=18001, D=4096, varlen=8),
        # FP32 throughout, two groups of B and C, 32 states per channel, no gate, odd length
        _scan("scan fp32 N32", B=2, T=1999, D=2048, N=32, G=2, io=FP32, z=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    io, st = rng.choice([(BF16, BF16), (BF16, FP32), (FP32, FP32)])
    kind = rng.choice(["tokens", "prompt", "packed"])
    more = dict(io=io, st=st, state=rng.random() < 0.7)
    if rng.random() < 0.4:
        C = 8 * _log(rng, 8, 4608)
        room = 8192 * 36864 // (C * (2 if io == FP32 else 1))  # tokens
        more.update(C=C, W=rng.choice([2, 3, 4, 4]), act=rng.random() < 0.8,
                    bias=rng.random() < 0.5, sliced=rng.random() < 0.3)
        if kind == "tokens":
            return _conv(B=_log(rng, 1, max(1, min(256, room))), T=rng.choice([1, 1, 1, 2, 5, 8]),
                         **dict(more, state=True), pool=rng.random() < 0.5)
        if kind == "prompt":
            T = _log(rng, 9, min(8192, room))
            return _conv(B=_log(rng, 1, max(1, min(32, room // T))), T=T, **more)
        T = _log(rng, 64, min(32768, room))
        return _conv(T=T, varlen=_log(rng, 1, max(1, min(64, T // 16))), **more)
    D = 8 * _log(rng, 8, 1024)
    N = rng.choice([8, 16, 16, 16, 32, 64])
    room = 8192 * 8192 * 16 // (D * N * (2 if io == FP32 else 1))
    more.update(D=D, N=N, G=rng.choice([1, 1, 2]) if D % 128 == 0 else 1, z=rng.random() < 0.7,
                skip=rng.random() < 0.8, softplus=rng.random() < 0.8)
    if kind == "tokens":
        return _scan(B=_log(rng, 1, max(1, min(256, 128 * 8192 * 16 // (D * N)))),
                     T=rng.choice([1, 1, 1, 2, 5, 8]), **dict(more, state=True),
                     pool=rng.random() < 0.5)
    if kind == "prompt":
        T = _log(rng, 9, min(8192, room))
        return _scan(B=_log(rng, 1, max(1, min(16, room // T))), T=T, **more)
    T = _log(rng, 64, min(16384, room))
    return _scan(T=T, varlen=_log(rng, 1, max(1, min(32, T // 16))), **more)


# ---------------------------------------------------------------- inputs


def _lengths(T, n, gen):
    """Offsets of n sequences that sum to T, uneven, from the generator."""
    w = 0.125 + torch.rand(n, generator=gen, dtype=torch.float64)
    cut = (torch.cumsum(w, 0) / w.sum() * T).round().to(torch.int64)
    cut[-1] = T
    return torch.cat([torch.zeros(1, dtype=torch.int64), cut])


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)

    def randn(*shape, dt=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dt)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    B, T = c["B"], c["T"]
    io, st = _dt(c["io"]), _dt(c["st"])
    s = {"case": c, "cu": None}
    N = c["varlen"] or B
    if c["varlen"]:
        s["cu"] = _lengths(T, N, cpu).to(dev)
        s["longest"] = int((s["cu"][1:] - s["cu"][:-1]).max())
    if c["op"] == "conv":
        C, W = c["C"], c["W"]
        # `sliced`: the first half of each row of a projection
        s["x"] = randn(B, T, 2 * C, dt=io)[..., :C] if c["sliced"] else randn(B, T, C, dt=io)
        s["weight"] = (2 * rand(C, W) - 1) * W ** -0.5
        s["bias"] = randn(C, scale=0.1) if c["bias"] else None
        slot, scale = (W - 1, C), 1.0
    else:
        D, n, G = c["D"], c["N"], c["G"]
        s["u"] = randn(B, T, D, dt=io)
        # step sizes between 1e-3 and 1e-1 for each channel, and what the token adds to them
        step = 1e-3 * 100 ** rand(D)
        if c["softplus"]:
            s["delta_bias"] = torch.log(torch.expm1(step))
            s["delta"] = randn(B, T, D, dt=io)
        else:
            s["delta_bias"] = None
            s["delta"] = (step * torch.exp(randn(B, T, D))).to(io)
        s["A"] = -torch.arange(1, n + 1, device=dev).float() * torch.exp(randn(D, n, scale=0.2))
        # B and C as the last parts of one projection, behind the step sizes' part
        parts = randn(B, T, 64 + 2 * G * n, dt=io)[..., 64:].unflatten(-1, (2, G, n))
        s["B"], s["C"] = parts[:, :, 0], parts[:, :, 1]
        s["D"] = 1 + randn(D, scale=0.1) if c["skip"] else None
        s["z"] = randn(B, T, D, dt=io) if c["z"] else None
        slot, scale = (D, n), 0.2
    if c["pool"]:
        s["pool"] = randn(2 * N + 3, *slot, dt=st, scale=scale)
        ids = torch.randperm(2 * N + 3, generator=cpu).to(torch.int32).to(dev)
        s["from"], s["to"] = ids[:N].contiguous(), ids[N:2 * N].contiguous()
    else:
        s["state"] = randn(N, *slot, dt=st, scale=scale) if c["state"] else None
    return s


# ---------------------------------------------------------------- the plain forms


def _start(s, slot):
    """The sequences' initial states in FP32."""
    c = s["case"]
    if c["pool"]:
        return s["pool"][s["from"].long()].float()
    if s["state"] is None:
        return torch.zeros(c["varlen"] or c["B"], *slot, device=torch.device("cuda"))
    return s["state"].float()


def _end(s, state):
    """The final states as the case keeps them: a tensor of their own, or the pool."""
    state = state.to(_dt(s["case"]["st"]))
    if s["case"]["pool"]:
        s["pool"][s["to"].long()] = state
        return s["pool"]
    return state


def _silu(x):
    return x / (1 + torch.exp(-x))


def _plain_conv(s):
    c = s["case"]
    W, T = c["W"], c["T"]
    x, w = s["x"].float(), s["weight"]
    state = _start(s, (W - 1, c["C"]))
    if c["varlen"]:
        token = torch.arange(T, device=x.device)
        seq = (token[:, None] >= s["cu"][1:]).sum(1).clamp(max=c["varlen"] - 1)
        begin, end = s["cu"][:-1], s["cu"][1:]

        def at(pos, n):
            """Input rows at positions pos of sequences n: before its begin, its state's."""
            rel = pos - begin[n]
            rows = x[0][pos.clamp(min=0, max=T - 1)]
            return torch.where((rel >= 0)[:, None], rows, state[n, (W - 1 + rel).clamp(0, W - 2)])

        y = sum(w[:, i] * at(token - (W - 1 - i), seq) for i in range(W))[None]
        all_ = torch.arange(c["varlen"], device=x.device)
        state = torch.stack([at(end - (W - 1 - i), all_) for i in range(W - 1)], 1)
    else:
        x = torch.cat([state, x], 1)
        y = sum(w[:, i] * x[:, i:i + T] for i in range(W))
        state = x[:, T:]
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["act"]:
        y = _silu(y)
    return y.to(s["x"].dtype), _end(s, state)


def _plain_scan(s):
    c = s["case"]
    T, D, n, G = c["T"], c["D"], c["N"], c["G"]
    u, delta, Bt, Ct = (s[k].float() for k in ("u", "delta", "B", "C"))
    if s["delta_bias"] is not None:
        delta = delta + s["delta_bias"]
    if c["softplus"]:
        delta = delta.clamp(min=0) + torch.log1p(torch.exp(-delta.abs()))
    N, longest = c["B"], T
    state = _start(s, (D, n))
    if c["varlen"]:  # one row for each sequence, zeros behind its end
        N, longest = c["varlen"], s["longest"]
        at = s["cu"][:-1, None] + torch.arange(longest, device=u.device)
        held = at < s["cu"][1:, None]
        rows = lambda x: x[0][at.clamp(max=T - 1)] * held.reshape(
            held.shape + (1,) * (x.dim() - 2))
        u, delta, Bt, Ct = rows(u), rows(delta), rows(Bt), rows(Ct)
    # chunks of L tokens, all at once: their end states from zero, then their start states one
    # after another, then the tokens again from those
    L = min(64, longest)
    P = (longest + L - 1) // L
    pad = lambda x: torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, P * L - longest)
                                            ).reshape(N, P, L, *x.shape[2:])
    u, delta, Bt, Ct = pad(u), pad(delta), pad(Bt), pad(Ct)
    x = delta * u
    A = s["A"]
    heads = lambda b: b.repeat_interleave(D // G, -2) if G > 1 else b  # [..., G or 1, n]

    def step(h, j):
        return torch.exp(delta[:, :, j, :, None] * A) * h + x[:, :, j, :, None] * heads(Bt[:, :, j])

    h = torch.zeros(N, P, D, n, device=u.device)
    if P > 1:
        for j in range(L):
            h = step(h, j)
        through = torch.exp(delta.double().sum(2).float()[..., None] * A)
        starts = [state]
        for p in range(P - 1):
            starts.append(through[:, p] * starts[-1] + h[:, p])
        h = torch.stack(starts, 1)
    else:
        h = state[:, None]
    y = torch.empty_like(u)
    for j in range(L):
        h = step(h, j)
        y[:, :, j] = (h * heads(Ct[:, :, j])).sum(-1)
    # zeros behind a sequence's end change no state: exp(0) h + 0
    final = h[:, P - 1]
    y = y.reshape(N, P * L, D)[:, :longest]
    y = y[held][None] if c["varlen"] else y
    if s["D"] is not None:
        y = y + s["D"] * s["u"].float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(s["u"].dtype), _end(s, final)


# ---------------------------------------------------------------- the package's calls


def _states(s):
    """How the package is given the case's states."""
    if s["case"]["pool"]:
        return dict(state_in=s["pool"], ssm_state_indices=s["from"], state_out_indices=s["to"])
    return dict(state_in=s["state"], state_dtype=_dt(s["case"]["st"]))


def _own_conv(s):
    import chunkwise_delta_rule_kda_amd as kda

    return kda.kda_short_conv(s["x"], s["weight"], s["bias"], cu_seqlens=s["cu"],
                              activation="silu" if s["case"]["act"] else None, **_states(s))


def _own_scan(s):
    import chunkwise_delta_rule_kda_amd as kda

    return kda.kda_selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                  cu_seqlens=s["cu"], delta_bias=s["delta_bias"],
                                  delta_softplus=s["case"]["softplus"], **_states(s))


def run(state):
    op = state["case"]["op"]
    if own:
        return {"conv": _own_conv, "scan": _own_scan}[op](state)
    return {"conv": _plain_conv, "scan": _plain_scan}[op](state)


# ---------------------------------------------------------------- work and exact values


def work(case):
    c = case
    tokens, N = c["B"] * c["T"], c["varlen"] or c["B"]
    io, st = _size(c["io"]), _size(c["st"])
    twice = 2 if c["pool"] or c["state"] else 1  # states read and written, or written
    if c["op"] == "conv":
        C, W = c["C"], c["W"]
        moved = 2 * io * tokens * C + st * N * (W - 1) * C * twice + 4 * C * (W + c["bias"])
        return {"bytes": moved, "flops": tokens * C * (2 * W + (4 if c["act"] else 0))}
    D, n, G = c["D"], c["N"], c["G"]
    moved = io * tokens * ((3 + c["z"]) * D + 2 * G * n) + st * N * D * n * twice
    moved += 4 * D * (n + c["skip"] + c["softplus"])
    # per state: the decay's exponent and exponential, its product, the write and the read-out
    return {"bytes": moved, "flops": 7 * tokens * D * n}


def _spans(c, s):
    if c["varlen"]:
        cu = s["cu"].tolist()
        return [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]
    return [(b, 0, c["T"]) for b in range(c["B"])]


def _exact_start(c, s, n, slot):
    if c["pool"]:
        return s["pool"][int(s["from"][n])].double()
    if s["state"] is None:
        return torch.zeros(*slot, dtype=torch.float64, device=torch.device("cuda"))
    return s["state"][n].double()


def _exact_end(c, s, ends):
    if not c["pool"]:
        return torch.stack(ends)
    pool = s["pool"].double()
    for n, slot in enumerate(s["to"].tolist()):
        pool[slot] = ends[n]
    return pool


def _exact_conv(c, s):
    """Each sequence's inputs behind its state's rows, every tap's product."""
    W = c["W"]
    w = s["weight"].double()
    out = torch.zeros(s["x"].shape, dtype=torch.float64, device=s["x"].device)
    ends = []
    for n, (b, lo, hi) in enumerate(_spans(c, s)):
        line = torch.cat([_exact_start(c, s, n, (W - 1, c["C"])), s["x"][b, lo:hi].double()])
        windows = line.unfold(0, W, 1)  # [tokens, C, W] (none for an empty sequence)
        y = (windows * w).sum(-1)[:hi - lo]
        if s["bias"] is not None:
            y = y + s["bias"].double()
        out[b, lo:hi] = y * torch.sigmoid(y) if c["act"] else y
        ends.append(line[hi - lo:])
    return out, _exact_end(c, s, ends)


def _exact_scan(c, s):
    """The definition, token after token; sequences side by side, the longest ones first."""
    D, n, G = c["D"], c["N"], c["G"]
    spans = _spans(c, s)
    lens = [hi - lo for _, lo, hi in spans]
    if max(lens) > 20000:
        return None
    order = sorted(range(len(spans)), key=lambda i: -lens[i])
    dev = s["u"].device
    flat = lambda t: t.reshape((-1,) + t.shape[2:])
    u, delta, Bt, Ct = flat(s["u"]), flat(s["delta"]), flat(s["B"]), flat(s["C"])
    first = torch.tensor([spans[i][0] * c["T"] + spans[i][1] for i in order], device=dev)
    S = torch.stack([_exact_start(c, s, i, (D, n)) for i in order])
    A = s["A"].double()
    y = torch.zeros(u.shape, dtype=torch.float64, device=dev)
    for t in range(max(lens)):
        k = sum(1 for m in lens if m > t)
        row = first[:k] + t
        d = delta[row].double()
        if s["delta_bias"] is not None:
            d = d + s["delta_bias"].double()
        if c["softplus"]:
            d = torch.logaddexp(d, torch.zeros_like(d))
        b, r = Bt[row].double(), Ct[row].double()  # [k, G, n]
        now = S[:k].view(k, G, D // G, n)
        now *= torch.exp(d[..., None] * A).view(k, G, D // G, n)
        now += (d * u[row].double()).view(k, G, D // G, 1) * b[:, :, None]
        y[row] = torch.matmul(now, r[..., None])[..., 0].reshape(k, D)
    y = y.view(s["u"].shape)
    if s["D"] is not None:
        y = y + s["D"].double() * s["u"].double()
    if s["z"] is not None:
        y = y * s["z"].double() * torch.sigmoid(s["z"].double())
    place = {i: j for j, i in enumerate(order)}
    return y, _exact_end(c, s, [S[place[i]] for i in range(len(spans))])


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_conv(case, s) if case["op"] == "conv" else _exact_scan(case, s)
