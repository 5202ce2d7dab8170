"""Cases of the per-head-decay linear attention, the state pool's slot operations and the
gated norm: their inputs, their plain forms in elementary torch operations, and the calls
of this package that compute the same.

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


def _linear(name=None, *, B=1, T=1, H=1, Hk=None, K=128, V=128, io=BF16, st=BF16, g=FP32,
            fixed=False, varlen=0, pool=False, state=True):
    """B sequences of T tokens (varlen: that many sequences packed into T tokens)."""
    c = dict(op="linear", B=B, T=T, H=H, Hk=Hk or H, K=K, V=V, io=io, st=st, g=g, fixed=fixed,
             varlen=varlen, pool=pool, state=state)
    return dict(c, name=name) if name else c


def _copy(name=None, *, slots, pairs, H, layers=1, fork=False, clear=0, src=BF16, dst=BF16):
    c = dict(op="copy", slots=slots, pairs=pairs, H=H, layers=layers, fork=fork, clear=clear,
             src=src, dst=dst)
    return dict(c, name=name) if name else c


def _compact(name=None, *, slots, live, moves, H, layers=1, dt=BF16):
    c = dict(op="compact", slots=slots, live=live, moves=moves, H=H, layers=layers, dt=dt)
    return dict(c, name=name) if name else c


def _norm(name=None, *, M, G, D, io=BF16, act="sigmoid", gate=True, residual=False, nxt=False,
          sliced=False):
    c = dict(op="norm", M=M, G=G, D=D, io=io, act=act, gate=gate, residual=residual, nxt=nxt,
             sliced=sliced)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's next token in a small layer: latency
        _linear("linear token H6", B=1, T=1, H=6),
        # a serving batch's next tokens: states read from their slots of an FP32 pool and
        # written to others (the first token after a fork), q/k heads shared by four
        _linear("linear tokens pool H24", B=128, T=1, H=24, Hk=6, st=FP32, pool=True),
        # a long prompt on few heads (a tensor-parallel shard)
        _linear("linear prompt H6", B=1, T=8192, H=6),
        # the same prompt on a whole layer
        _linear("linear prompt H96", B=1, T=8192, H=96),
        # a packed batch of prompts with initial states kept in FP32
        _linear("linear packed H24", T=18001, H=24, varlen=8, st=FP32),
        # FP32 throughout, a fixed decay for each head, odd length
        _linear("linear fp32 fixed H12", B=2, T=1999, H=12, io=FP32, st=FP32, fixed=True),
        # one state forked to four for sampling in parallel
        _copy("pool fork 1 to 4", slots=16, pairs=4, H=6, fork=True),
        # stored FP32 prefix states brought into the slots of a BF16 pool of several layers
        _copy("pool restore 48", slots=96, pairs=48, H=24, layers=4, clear=3, src=FP32),
        # a small pool tidied after a few sequences ended
        _compact("pool compact 64", slots=64, live=40, moves=9, H=6),
        # a large pool halved so that its upper part can be given back
        _compact("pool compact 512", slots=512, live=200, moves=120, H=24, layers=2, dt=FP32),
        # heads' outputs of a serving batch normed and gated, gate a slice of a projection
        _norm("norm heads 64 tokens", M=64, G=24, D=128, sliced=True),
        # between two blocks of a wide model: norm, gate, residual scale and next norm
        _norm("norm block 8192", M=8192, G=1, D=12288, act="silu", residual=True, nxt=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "copy", "compact", "norm"])
    if op == "linear":
        H = _log(rng, 1, 96)
        Hk = rng.choice([d for d in range(1, H + 1) if H % d == 0])
        io, st = rng.choice([(BF16, BF16), (BF16, FP32), (FP32, FP32)])
        K, V = rng.choice([64, 128, 128]), rng.choice([64, 128, 128, 256])
        kind = rng.choice(["tokens", "prompt", "packed"])
        room = 8192 * 96 * 128 // (H * max(K, V) * (3 if io == FP32 else 1))  # tokens
        more = dict(H=H, Hk=Hk, K=K, V=V, io=io, st=st, g=rng.choice([io, FP32]),
                    state=rng.random() < 0.7)
        if kind == "tokens":
            return _linear(B=_log(rng, 1, max(1, min(256, 3000 // H))), T=rng.choice([1, 1, 1, 2, 5, 8]),
                           fixed=rng.random() < 0.3, **dict(more, state=True),
                           pool=rng.random() < 0.5)
        if kind == "prompt":
            T = _log(rng, 9, min(8192, room))
            return _linear(B=_log(rng, 1, max(1, min(32, room // T, 1000 // H))), T=T,
                           fixed=rng.random() < 0.3, **more)
        T = _log(rng, 64, min(16384, room))
        return _linear(T=T, varlen=_log(rng, 1, max(1, min(64, T // 16, 1000 // H))), **more)
    if op == "copy":
        H, layers = _log(rng, 1, 48), rng.choice([1, 1, 2, 5])
        pairs = _log(rng, 1, max(1, min(128, 4608 // (H * layers))))
        return _copy(slots=2 * pairs + rng.randrange(1, 9), pairs=pairs, H=H, layers=layers,
                     fork=rng.random() < 0.4, clear=rng.randrange(0, 1 + pairs // 4),
                     src=rng.choice([BF16, FP32]), dst=rng.choice([BF16, FP32]))
    if op == "compact":
        H, layers = _log(rng, 1, 48), rng.choice([1, 1, 3])
        slots = _log(rng, 8, max(8, min(512, 14000 // (H * layers))))
        live = rng.randrange(1, slots)
        return _compact(slots=slots, live=live, moves=rng.randrange(0, 1 + min(live, slots - live)),
                        H=H, layers=layers, dt=rng.choice([BF16, FP32]))
    D = 8 * _log(rng, 8, 1536) if rng.random() < 0.5 else rng.choice([64, 128])
    G = 1 if D > 128 else _log(rng, 1, 96)
    return _norm(M=_log(rng, 1, max(1, min(8192, 8192 * 6000 // (D * G)))), G=G, D=D,
                 io=rng.choice([BF16, FP32]), act=rng.choice(["sigmoid", "silu"]),
                 gate=rng.random() < 0.8, residual=rng.random() < 0.5, nxt=rng.random() < 0.5,
                 sliced=rng.random() < 0.3)


# ---------------------------------------------------------------- inputs


def _lengths(T, n, gen):
    """n lengths that sum to T, uneven, from the generator."""
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

    s = {"case": c}
    if c["op"] == "linear":
        B, T, H, Hk, K, V = (c[n] for n in ("B", "T", "H", "Hk", "K", "V"))
        io, st = _dt(c["io"]), _dt(c["st"])
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)
        s["q"] = unit(randn(B, T, Hk, K)).to(io)
        s["k"] = unit(randn(B, T, Hk, K)).to(io)
        s["v"] = randn(B, T, H, V, dt=io)
        rate = 0.02 * 50 ** torch.rand(H, generator=gen, device=dev)  # heads of 50 to 1 tokens' memory
        s["log_decay"] = -rate if c["fixed"] else None
        s["g"] = None if c["fixed"] else (
            -rate * torch.nn.functional.softplus(randn(B, T, H))).to(_dt(c["g"]))
        N = B
        s["cu"] = None
        if c["varlen"]:
            N = c["varlen"]
            s["cu"] = _lengths(T, N, cpu).to(dev)
            s["longest"] = int((s["cu"][1:] - s["cu"][:-1]).max())
        if c["pool"]:
            s["pool"] = randn(2 * N + 3, H, V, K, dt=st, scale=0.1)
            ids = torch.randperm(2 * N + 3, generator=cpu).to(torch.int32).to(dev)
            s["from"], s["to"] = ids[:N].contiguous(), ids[N:2 * N].contiguous()
        else:
            s["state"] = randn(N, H, V, K, dt=st, scale=0.1) if c["state"] else None
    elif c["op"] == "copy":
        P, L = c["pairs"], c["layers"]
        shape = (L, c["slots"], c["H"], 128, 128)
        s["pool"] = randn(*shape, dt=_dt(c["dst"]))
        # a fork stays in its pool; a restore reads another one
        s["source"] = s["pool"] if c["fork"] and c["src"] == c["dst"] else randn(
            *shape, dt=_dt(c["src"]))
        ids = torch.randperm(c["slots"], generator=cpu).to(torch.int32)
        src, dst = ids[:P].clone(), ids[P:2 * P].clone()
        if c["fork"]:
            src[:] = src[0]
        src[P - c["clear"]:] = -1  # freed slots: zeros
        s["src"], s["dst"] = src.to(dev), dst.to(dev)
    elif c["op"] == "compact":
        n, live, moves = c["slots"], c["live"], c["moves"]
        low = torch.randperm(live, generator=cpu)[:live - moves]
        high = live + torch.randperm(n - live, generator=cpu)[:moves]
        ids = torch.cat([low, high])[torch.randperm(live, generator=cpu)]
        s["ids"] = ids.to(torch.int32).to(dev)
        s["pool"] = randn(c["layers"], n, c["H"], 128, 128, dt=_dt(c["dt"]))
    else:
        M, G, D = c["M"], c["G"], c["D"]
        io = _dt(c["io"])
        s["x"] = randn(M, G, D, dt=io)
        s["gate"] = None
        if c["gate"]:  # `sliced`: the last of three projections held in one tensor
            s["gate"] = randn(M, 3, G, D, dt=io)[:, 2] if c["sliced"] else randn(M, G, D, dt=io)
        s["weight"] = 1 + randn(D, scale=0.1)
        s["residual"] = randn(M, G, D, dt=io) if c["residual"] else None
        s["next"] = 1 + randn(D, scale=0.1) if c["nxt"] else None
    return s


# ---------------------------------------------------------------- the plain forms


def _plain_chunks(q, k, v, g, state, scale):
    """q, k [N, T, H, K], v [N, T, H, V] in FP32, g [N, T, H] in FP64 (sums of log decays are
    subtracted from each other), state [N, H, V, K]: all chunks at once."""
    N, T, H, K = q.shape
    V = v.shape[-1]
    C = min(64, T)
    P = (T + C - 1) // C
    pad = P * C - T
    cut = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).reshape(
        N, P, C, H, x.shape[-1]).permute(0, 3, 1, 2, 4).reshape(N * H * P, C, x.shape[-1])
    q, k, v = cut(q), cut(k), cut(v)
    g = cut(g[..., None]).reshape(N * H, P, C)
    G = torch.cumsum(g, -1)
    tri = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    near = (G[..., :, None] - G[..., None, :]).masked_fill(~tri, -float("inf"))
    near = torch.exp(near).float().reshape(N * H * P, C, C)
    inner = torch.bmm(torch.bmm(q, k.transpose(1, 2).contiguous()) * near, v)
    end = torch.exp(G[..., -1:] - G).float().reshape(N * H * P, C, 1)
    Z = torch.bmm((v * end).transpose(1, 2).contiguous(), k).reshape(N * H, P, V * K)
    # start state of chunk p: the first state and the Z of the chunks before, decayed
    S = torch.cumsum(torch.cat([torch.zeros_like(G[:, :1, -1]), G[..., -1]], 1), 1)
    far = S[:, :, None] - S[:, None, :]
    tri = torch.ones(P + 1, P + 1, dtype=torch.bool, device=q.device).tril()
    far = torch.exp(far.masked_fill(~tri, -float("inf"))).float()
    states = torch.bmm(far, torch.cat([state.reshape(N * H, 1, V * K), Z], 1))
    first = states[:, :P].reshape(N * H * P, V, K)
    outer = torch.bmm(q, first.transpose(1, 2).contiguous())
    outer = outer * torch.exp(G).float().reshape(N * H * P, C, 1)
    o = scale * (inner + outer)
    o = o.reshape(N, H, P * C, V)[:, :, :T].permute(0, 2, 1, 3)
    return o, states[:, P].reshape(N, H, V, K)


def _plain_linear(s):
    c = s["case"]
    H, V, K = c["H"], c["V"], c["K"]
    q, k = (s[n].float().repeat_interleave(H // c["Hk"], 2) for n in ("q", "k"))
    v = s["v"].float()
    if s["g"] is None:
        g = s["log_decay"].double().expand(c["B"], c["T"], H)
    else:
        g = s["g"].double()
    N = c["varlen"] or c["B"]
    if c["varlen"]:  # one row for each sequence, zeros behind its end
        at = s["cu"][:-1, None] + torch.arange(s["longest"], device=q.device)
        held = at < s["cu"][1:, None]
        rows = lambda x: x[0][at.clamp(max=c["T"] - 1)] * held.reshape(
            held.shape + (1,) * (x.dim() - 2)).to(x.dtype)
        q, k, v, g = rows(q), rows(k), rows(v), rows(g)
    if c["pool"]:
        state = s["pool"][s["from"].long()].float()
    elif s["state"] is None:
        state = torch.zeros(N, H, V, K, device=q.device)
    else:
        state = s["state"].float()
    o, state = _plain_chunks(q, k, v, g, state, K ** -0.5)
    if c["varlen"]:
        o = o[held][None]
    o, state = o.to(s["v"].dtype).contiguous(), state.to(_dt(c["st"]))
    if c["pool"]:
        s["pool"][s["to"].long()] = state
        state = s["pool"]
    return o, state


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    held = (src >= 0)[None, :, None, None, None]
    rows = s["source"][:, src.clamp(min=0)].to(s["pool"].dtype)
    s["pool"][:, dst] = torch.where(held, rows, torch.zeros_like(rows))
    return s["pool"]


def _plain_compact(s):
    pool, ids = s["pool"], s["ids"].long()
    n = pool.shape[1]
    live = torch.zeros(n, dtype=torch.int64, device=ids.device)
    live[ids] = 1
    count = live.sum()
    slot = torch.arange(n, device=ids.device)
    free = ((live == 0) & (slot < count)).long()
    late = ((live == 1) & (slot >= count)).long()
    # the k-th late slot goes to the k-th free one
    order = torch.argsort(free, descending=True, stable=True)
    new = torch.where(late == 1, order[(torch.cumsum(late, 0) - 1).clamp(min=0)], slot)[ids]
    # entries that stay repeat the first move, or the first entry's stay where none moves
    first = torch.argmax((new != ids).long())
    moved = new != ids
    a, b = torch.where(moved, ids, ids[first]), torch.where(moved, new, new[first])
    pool[:, b] = pool[:, a]
    return pool, new.to(torch.int32), count.to(torch.int32).reshape(1)


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s["weight"]
    if s["gate"] is not None:
        e = s["gate"].float()
        a = 1 / (1 + torch.exp(-e))
        y = y * (e * a if c["act"] == "silu" else a)
    y = 0.5 * y
    if s["residual"] is not None:
        y = s["residual"].float() + y
    if s["next"] is None:
        return y.to(s["x"].dtype)
    z = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * s["next"]
    return y.to(s["x"].dtype), z.to(s["x"].dtype)


# ---------------------------------------------------------------- the package's calls


def _own_linear(s):
    import chunkwise_delta_rule_kda_amd as kda

    if s["case"]["pool"]:
        return kda.kda_linear(s["q"], s["k"], s["v"], s["g"], s["pool"],
                              log_decay=s["log_decay"], ssm_state_indices=s["from"],
                              state_out_indices=s["to"])
    return kda.kda_linear(s["q"], s["k"], s["v"], s["g"], s["state"], s["cu"],
                          log_decay=s["log_decay"], state_dtype=_dt(s["case"]["st"]))


def _own_copy(s):
    import chunkwise_delta_rule_kda_amd as kda

    return kda.kda_pool_copy(s["pool"], s["src"], s["dst"], source=s["source"], layered=True)


def _own_compact(s):
    import chunkwise_delta_rule_kda_amd as kda

    ids, count = kda.kda_pool_compact(s["pool"], s["ids"], layered=True)
    return s["pool"], ids, count


def _own_norm(s):
    import chunkwise_delta_rule_kda_amd as kda

    return kda.kda_gated_norm(s["x"], s["gate"], s["weight"], s["residual"],
                              next_weight=s["next"], gate_act=s["case"]["act"], scale=0.5)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _own_linear, "copy": _own_copy, "compact": _own_compact,
                "norm": _own_norm}[op](state)
    return {"linear": _plain_linear, "copy": _plain_copy, "compact": _plain_compact,
            "norm": _plain_norm}[op](state)


# ---------------------------------------------------------------- work and exact values


def work(case):
    c = case
    if c["op"] == "linear":
        tokens, N = c["B"] * c["T"], c["varlen"] or c["B"]
        io, st = _size(c["io"]), _size(c["st"])
        moved = io * tokens * (2 * c["Hk"] * c["K"] + 2 * c["H"] * c["V"])
        moved += 0 if c["fixed"] else tokens * c["H"] * _size(c["g"])
        moved += st * N * c["H"] * c["V"] * c["K"] * (2 if c["pool"] or c["state"] else 1)
        # the recurrence itself: an outer product into the state and a product with it
        return {"bytes": moved, "flops": 4 * tokens * c["H"] * c["K"] * c["V"]}
    if c["op"] == "copy":
        slot = c["layers"] * c["H"] * 128 * 128
        read = 1 if c["fork"] else c["pairs"] - c["clear"]
        return {"bytes": slot * (_size(c["src"]) * read + _size(c["dst"]) * c["pairs"]), "flops": 0}
    if c["op"] == "compact":
        moved = 2 * c["moves"] * c["layers"] * c["H"] * 128 * 128 * _size(c["dt"])
        return {"bytes": moved + 8 * c["live"] + 4, "flops": 0}
    n = c["M"] * c["G"] * c["D"]
    tensors = 2 + c["gate"] + c["residual"] + c["nxt"]
    return {"bytes": tensors * n * _size(c["io"]) + 4 * c["D"] * (1 + c["nxt"]), "flops": 10 * n}


def _exact_linear(c, s):
    """The definition, token after token."""
    dev, f64 = s["q"].device, torch.float64
    H, V, K = c["H"], c["V"], c["K"]
    group = H // c["Hk"]
    if c["varlen"]:
        cu = s["cu"].tolist()
        starts, lens = cu[:-1], [b - a for a, b in zip(cu[:-1], cu[1:])]
    else:
        starts, lens = [b * c["T"] for b in range(c["B"])], [c["T"]] * c["B"]
    N = len(lens)
    flat = lambda x: x.reshape((-1,) + x.shape[2:])
    q, k, v = flat(s["q"]), flat(s["k"]), flat(s["v"])
    g = None if s["g"] is None else flat(s["g"])
    if c["pool"]:
        S = s["pool"].index_select(0, s["from"].long()).to(f64)
    elif s["state"] is not None:
        S = s["state"].to(f64)
    else:
        S = torch.zeros(N, H, V, K, dtype=f64, device=dev)
    o = torch.zeros(v.shape, dtype=f64, device=dev)
    # sequences from the longest to the shortest: those that still run are a front part
    order = sorted(range(N), key=lambda n: -lens[n])
    S = S[torch.tensor(order, device=dev)]
    start = torch.tensor([starts[n] for n in order], device=dev)
    decay = None if s["log_decay"] is None else torch.exp(s["log_decay"].to(f64))
    for t in range(max(lens)):
        n = sum(1 for m in lens if m > t) if c["varlen"] else N
        row = start[:n] + t
        kt = k[row].to(f64).repeat_interleave(group, 1)
        qt = q[row].to(f64).repeat_interleave(group, 1)
        d = decay[None].expand(n, H) if g is None else torch.exp(g[row].to(f64))
        A = S[:n]
        A *= d[..., None, None]
        A += v[row].to(f64)[..., None] * kt[:, :, None]
        o[row] = torch.matmul(A, qt[..., None])[..., 0] * K ** -0.5
    back = torch.empty(N, dtype=torch.int64)
    back[torch.tensor(order)] = torch.arange(N)
    S = S[back.to(dev)]
    if c["pool"]:
        pool = s["pool"].to(f64)
        pool.index_copy_(0, s["to"].long(), S)
        S = pool
    return o.reshape(s["v"].shape), S


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "linear":
        return _exact_linear(c, s)
    if c["op"] == "copy":
        source = s["source"]
        out = s["pool"].double()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            out[:, b] = source[:, a].double() if a >= 0 else 0.0
        return out
    if c["op"] == "compact":
        ids = s["ids"].tolist()
        count = len(set(ids))
        holes = [i for i in range(count) if i not in set(ids)]
        to = dict(zip(sorted(i for i in set(ids) if i >= count), holes))
        out = s["pool"].double()
        for a, b in to.items():
            out[:, b] = out[:, a]
        new = torch.tensor([to.get(i, i) for i in ids], dtype=torch.int32, device=out.device)
        return out, new, torch.tensor([count], dtype=torch.int32, device=out.device)
    x = s["x"].double()
    y = 0.5 * s["weight"].double() * x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    if s["gate"] is not None:
        e = s["gate"].double()
        y = y * torch.sigmoid(e)
        if c["act"] == "silu":
            y = y * e
    if s["residual"] is not None:
        y = y + s["residual"].double()
    if s["next"] is None:
        return y
    return y, s["next"].double() * y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6)
