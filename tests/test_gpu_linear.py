"""Linear attention with one decay per head (kda_linear) against the FP64 token recurrence.

Tolerances, element by element. With a = the oracle's sum of absolute terms and u = 2^-8
(half a BF16 step):
* o of BF16 calls: its own rounding, u |o|; every term passes at most two BF16 roundings
  (the decayed value written to a BF16-output state, then the state or the score as a
  matrix operand): 2 u a. FP32 sums and decay factors: e a, see below.
* the state: u |S| for a BF16 output, u a for the rounding of the decayed values, which
  FP32 outputs do not have (theirs are split into parts).
* FP32 arithmetic: a sum of n terms is off by at most n 2^-24 of its absolute terms. A
  chunk sums 64 tokens and K keys, and each of the T / 64 chunks adds a decay (exp2 of a
  rounded exponent: below 2^-24 (2 + |x|) relative, and |x| 2^-x <= 0.54, so 3 2^-24 of the
  undecayed term) and a product: e = (K + 64 + 8 (T / 64 + 2)) 2^-24. The split values
  leave 2^-24 of a term (three parts of eight bits).
"""

import numpy as np
import pytest

from oracle import linear_recurrence_fp64

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import chunkwise_delta_rule_kda_amd as kda

    kda.load_library()


def inputs(B, T, H, Hk=None, K=128, V=128, io="bf16", st="bf16", g="g", lens=None, seed=0,
           state=True, decay=1.0):
    """Device tensors; g: "g" per token FP32, "io" per token in the I/O type, "fixed" per
    head, "both", or None."""
    import torch

    Hk = Hk or H
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000 + seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp(min=1e-6)
    d = dict(q=unit(r(B, T, Hk, K)).to(dt[io]), k=unit(r(B, T, Hk, K)).to(dt[io]),
             v=r(B, T, H, V).to(dt[io]), g=None, log_decay=None, cu_seqlens=None,
             state_in=None)
    rate = decay * 0.02 * 50 ** torch.rand(H, generator=gen, device="cuda")
    if g in ("g", "io", "both"):
        x = -rate * torch.nn.functional.softplus(r(B, T, H))
        d["g"] = x.to(dt[io]) if g == "io" else x
    if g in ("fixed", "both"):
        d["log_decay"] = -rate
    N = B
    if lens is not None:
        d["cu_seqlens"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device="cuda",
                                       dtype=torch.int64)
        N = len(lens)
    d["state_dtype"] = dt[st]
    if state:
        d["state_in"] = (0.3 * r(N, H, V, K)).to(dt[st])
    return d


def host(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def oracle(d, state0=None, scale=None):
    cu = None if d["cu_seqlens"] is None else d["cu_seqlens"].cpu().numpy()
    return linear_recurrence_fp64(host(d["q"]), host(d["k"]), host(d["v"]), host(d["g"]),
                                  host(d["state_in"]) if state0 is None else state0,
                                  log_decay=host(d["log_decay"]), cu_seqlens=cu, scale=scale)


def fp32_part(T, K):
    return (K + 64 + 8 * (T / 64 + 2)) * 2.0 ** -24


def within(got, ref, slack, name):
    assert got.shape == ref.shape, name
    assert np.all(np.isfinite(got)), name
    over = np.abs(got - ref) - slack
    at = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    worst = np.max(np.abs(got - ref) / np.maximum(slack, 1e-300)) if over.size else 0.0
    print(f"[case] {name}: largest error is {worst:.3f} of its bound", flush=True)
    assert not over.size or over[at] <= 0, (name, at, got[at], ref[at], slack[at])


def check(o, s, ref, d, name):
    import torch

    o_ref, s_ref, o_abs, s_abs = ref
    T, K = d["q"].shape[1], d["q"].shape[3]
    e = fp32_part(T, K)
    bf16 = d["q"].dtype == torch.bfloat16
    within(host(o), o_ref, (U * np.abs(o_ref) + (2 * U + e) * o_abs) if bf16 else e * o_abs,
           name + " o")
    if s is not None:
        bf16_state = s.dtype == torch.bfloat16
        own = U * np.abs(s_ref) if bf16_state else 0.0
        term = U if bf16 and bf16_state else 2.0 ** -24 if bf16 else 0.0
        within(host(s), s_ref, own + (term + e) * s_abs, name + " state")


def run(d, **kw):
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    d = dict(d)
    q, k, v, g = (d.pop(n) for n in "qkvg")
    d.update(kw)
    out = kda.kda_linear(q, k, v, g, **d)
    torch.cuda.synchronize()
    return out


CASES = [
    # B, T, H, Hk, K, V, io, st, g
    (1, 64, 1, 1, 128, 128, "bf16", "bf16", "g"),      # one whole chunk
    (2, 1, 3, 1, 128, 128, "bf16", "bf16", "g"),       # one token by the chunked form
    (1, 63, 2, 2, 128, 128, "bf16", "fp32", "io"),
    (1, 65, 2, 1, 128, 128, "bf16", "bf16", "fixed"),
    (3, 130, 4, 2, 64, 64, "bf16", "fp32", "g"),
    (1, 200, 2, 1, 64, 128, "bf16", "bf16", "both"),
    (2, 100, 3, 3, 128, 64, "bf16", "bf16", "g"),
    (1, 129, 2, 2, 128, 256, "bf16", "fp32", None),    # no decay at all
    (1, 70, 2, 1, 128, 192, "bf16", "bf16", "g"),      # an odd number of value blocks
    (1, 65, 1, 1, 64, 512, "bf16", "bf16", "g"),
    (2, 97, 3, 1, 128, 128, "fp32", "fp32", "g"),
    (1, 130, 2, 2, 64, 64, "fp32", "bf16", "fixed"),
    (1, 64, 2, 2, 128, 192, "fp32", "fp32", "io"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_chunked_form(case):
    B, T, H, Hk, K, V, io, st, g = case
    d = inputs(B, T, H, Hk, K, V, io, st, g)
    o, s = run(d, segment_tokens=-1)
    check(o, s, oracle(d), d, f"serial {case}")


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_segments(case):
    B, T, H, Hk, K, V, io, st, g = case
    d = inputs(B, 3 * T + 5, H, Hk, K, V, io, st, g, seed=1)
    o, s = run(d, segment_tokens=64)
    check(o, s, oracle(d), d, f"segments {case}")


@pytest.mark.parametrize("T", [1, 2, 7, 8])
@pytest.mark.parametrize("B,H,Hk,K,V,io,st,g", [
    (1, 1, 1, 128, 128, "bf16", "bf16", "g"),
    (5, 3, 1, 128, 64, "bf16", "fp32", "io"),
    (3, 4, 2, 64, 128, "bf16", "bf16", "fixed"),
    (2, 2, 2, 64, 64, "fp32", "fp32", "both"),
    (4, 40, 8, 128, 128, "bf16", "bf16", "g"),          # more rows per workgroup
    (40, 8, 4, 128, 192, "fp32", "fp32", None),
    (70, 8, 8, 64, 256, "bf16", "fp32", "g"),
])
def test_token_form(T, B, H, Hk, K, V, io, st, g):
    d = inputs(B, T, H, Hk, K, V, io, st, g, seed=2)
    o, s = run(d)
    check(o, s, oracle(d), d, f"tokens T={T} B={B} H={H}")
    if B * H <= 8:  # and the chunked form of the same call
        o2, s2 = run(d, segment_tokens=-1)
        check(o2, s2, oracle(d), d, f"tokens, chunked T={T} B={B} H={H}")


@pytest.mark.parametrize("lens", [[5], [0, 64, 0, 1, 130, 0], [63, 65, 1, 1, 200, 128, 64],
                                  [1] * 70, [3, 0] * 40, [0, 0, 0]])
@pytest.mark.parametrize("seg", [0, -1, 64, 128])
def test_packed(lens, seg):
    T = sum(lens)
    for io, st in (("bf16", "bf16"), ("bf16", "fp32")):
        d = inputs(1, T, 2, 1, 128, 128, io, st, "g", lens=lens, seed=3)
        o, s = run(d, segment_tokens=seg)
        check(o, s, oracle(d), d, f"packed {len(lens)} of {T} seg {seg} {st}")
        if T == 0:
            assert s.equal(d["state_in"])


def test_packed_many_sequences():
    # more than 64 x 64 sequences: three levels of the search for a workgroup's sequence
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 3, 4500)
    d = inputs(1, int(lens.sum()), 1, 1, 64, 64, "bf16", "fp32", "g", lens=list(lens), seed=4)
    for seg in (-1, 64):
        o, s = run(d, segment_tokens=seg)
        check(o, s, oracle(d), d, f"packed 4500 seg {seg}")


def test_no_state_and_no_output_state():
    d = inputs(2, 150, 2, 2, 128, 128, "bf16", "bf16", "g", state=False)
    for seg in (-1, 64):
        o, s = run(d, segment_tokens=seg, output_final_state=False)
        assert s is None
        check(o, None, oracle(d), d, f"no states seg {seg}")
    d = inputs(2, 3, 2, 2, 128, 128, "bf16", "bf16", "g", state=False)
    o, s = run(d)
    check(o, s, oracle(d), d, "tokens from zero")


@pytest.mark.parametrize("T,seg", [(8, 0), (150, -1), (300, 64)])
def test_in_place_state(T, seg):
    d = inputs(2, T, 3, 1, 128, 128, "bf16", "fp32", "g", seed=6)
    ref = oracle(d)
    o, s = run(d, state_out=d["state_in"], segment_tokens=seg)
    assert s.data_ptr() == d["state_in"].data_ptr()
    check(o, s, ref, d, f"in place T={T}")


@pytest.mark.parametrize("T,seg", [(1, 0), (5, 0), (100, -1), (300, 64)])
@pytest.mark.parametrize("st", ["bf16", "fp32"])
def test_pool(T, seg, st):
    import torch

    B, H, V, K = 5, 2, 128, 128
    d = inputs(B, T, H, 1, K, V, "bf16", st, "g", seed=7, state=False)
    base = torch.randn(9, 2 * H, V, K, device="cuda").to(d["state_dtype"])
    pool = base[:, :H]  # padded slots
    frozen = base.clone()
    # a shared prefix (slot 2 read twice), an id out of range read, one out of range written
    src = torch.tensor([2, 2, 7, -1, 4], dtype=torch.int32, device="cuda")
    dst = torch.tensor([0, 1, 7, 3, 9], dtype=torch.int32, device="cuda")
    s0 = np.zeros((B, H, V, K))
    for n, i in enumerate(src.tolist()):
        if i >= 0:
            s0[n] = host(pool[i])
    ref = oracle(d, s0)
    o, s = run(d, state_in=pool, ssm_state_indices=src, state_out_indices=dst,
               segment_tokens=seg)
    assert s is pool
    held = [n for n, i in enumerate(dst.tolist()) if i < 9]
    got = torch.stack([pool[dst[n]] for n in held])
    pick = lambda x: x[held]
    check(o, got, (ref[0], pick(ref[1]), ref[2], pick(ref[3])), d, f"pool T={T} seg {seg} {st}")
    for i in range(9):
        if i not in dst.tolist():
            assert torch.equal(base[i], frozen[i]), i
        assert torch.equal(base[i, H:], frozen[i, H:]), i
    # without state_out_indices the slots read are written
    base.copy_(frozen)
    ids = torch.tensor([8, 0, 3, 5, 1], dtype=torch.int32, device="cuda")
    ref = oracle(d, np.stack([host(pool[i]) for i in ids.tolist()]))
    o, _ = run(d, state_in=pool, ssm_state_indices=ids, segment_tokens=seg)
    check(o, pool[ids.long()], ref, d, f"pool in place T={T} seg {seg} {st}")


@pytest.mark.parametrize("T,seg", [(3, 0), (200, -1), (200, 64)])
@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_strided_inputs(T, seg, io):
    """q, k, v as slices of one projection, heads before tokens, and repeated heads."""
    import torch

    B, H, K = 2, 3, 64
    d = inputs(B, T, H, H, K, K, io, "fp32", "g", seed=8)
    ref = oracle(d)
    packed = torch.full((B, T, 3, H, K + 8), float("nan"), device="cuda").to(d["q"].dtype)
    for i, n in enumerate("qkv"):
        packed[:, :, i, :, :K] = d[n]
        d[n] = packed[:, :, i, :, :K]
    o, s = run(d, segment_tokens=seg)
    check(o, s, ref, d, f"projection slices T={T}")
    for n in "qkv":  # [B, H, T, K] seen as [B, T, H, K]
        d[n] = d[n].transpose(1, 2).contiguous().transpose(1, 2)
    o, s = run(d, segment_tokens=seg)
    check(o, s, ref, d, f"heads before tokens T={T}")
    one = d["k"][:, :, :1]
    d["k"] = one.expand(B, T, H, K)
    ref = oracle(dict(d, k=one.expand(B, T, H, K).contiguous()))
    o, s = run(d, segment_tokens=seg)
    check(o, s, ref, d, f"one key row for all heads T={T}")


@pytest.mark.parametrize("seg", [-1, 64])
@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_emptied_states(seg, io):
    """Log decays of -inf, of the type's lowest value and of 0 between ordinary ones."""
    import torch

    for T in (6, 200):
        d = inputs(1, T, 2, 2, 128, 128, io, "fp32", "g", seed=9)
        low = torch.finfo(torch.float32).min
        d["g"][0, 3, 0] = -float("inf")
        d["g"][0, 4, 1] = low
        if T > 6:
            d["g"][0, 64, 0] = -float("inf")       # first token of a chunk
            d["g"][0, 127, 1] = -float("inf")      # last token of a chunk
            d["g"][0, 129:133] = low
            d["g"][0, 140:190] = 0.0
            d["g"][0, 190] = -60.0
        ref = oracle(d)
        o, s = run(d, segment_tokens=seg if T > 6 else 0)
        check(o, s, ref, d, f"emptied T={T} seg {seg}")


def test_strong_decay_keeps_near_tokens_exact():
    # 64 tokens of log decay -30 each: the prefix sums reach -1920, whose differences an
    # FP32 prefix would give to 1e-4 only
    d = inputs(1, 190, 1, 1, 128, 128, "fp32", "fp32", "g", seed=10)
    d["g"][:] = -30.0
    d["g"][0, 1::2] = -0.01
    o, s = run(d, segment_tokens=-1)
    check(o, s, oracle(d), d, "strong decay")


def test_bad_values_stay_in_their_sequence_and_head():
    import torch

    lens = [70, 70, 70]
    d = inputs(1, 210, 2, 2, 128, 128, "bf16", "fp32", "g", lens=lens, seed=11)
    ref = oracle(d)
    d["v"][0, 100, 1] = float("nan")
    d["k"][0, 130, 1, 5] = float("inf")
    o, s = run(d, segment_tokens=-1)
    o[0, 70:140, 1] = 0
    s[1, 1] = 0
    for a in (ref[0], ref[2]):
        a[0, 70:140, 1] = 0
    for a in (ref[1], ref[3]):
        a[1, 1] = 0
    check(o, s, ref, dict(d, k=d["k"].nan_to_num(0, 0, 0)), "bad values")


def test_rows_behind_the_tensor_are_not_touched():
    """Outputs inside a larger buffer: nothing is written outside [B, T, H, V]."""
    import torch

    for io in ("bf16", "fp32"):
        d = inputs(1, 67, 2, 1, 64, 64, io, "fp32", "g", seed=12)
        big = torch.full((80 * 2 * 64,), 7.0, device="cuda").to(d["q"].dtype)
        n = 67 * 2 * 64
        o = big[256:256 + n].view(1, 67, 2, 64)
        o2, s = run(d, o=o, segment_tokens=-1)
        check(o2, s, oracle(d), d, "inside a buffer")
        assert bool((big[:256] == 7).all()) and bool((big[256 + n:] == 7).all())


def test_empty_calls():
    import torch

    d = inputs(2, 0, 3, 1, 128, 128, "bf16", "fp32", "g", seed=13)
    o, s = run(d)
    assert o.shape == (2, 0, 3, 128) and torch.equal(s, d["state_in"])
    d = inputs(2, 0, 3, 1, 128, 128, "bf16", "bf16", "g", state=False)
    o, s = run(d)
    assert not s.any()


def test_scale():
    d = inputs(1, 80, 2, 2, 128, 128, "fp32", "fp32", "g", seed=14)
    o, s = run(d, scale=0.37, segment_tokens=64)
    check(o, s, oracle(d, scale=float(np.float32(0.37))), d, "scale")


@pytest.mark.parametrize("T,seg", [(4, 0), (200, -1), (200, 64)])
def test_results_are_the_same_every_time(T, seg):
    import torch

    d = inputs(2, T, 3, 1, 128, 128, "bf16", "fp32", "g", seed=15)
    o, s = run(d, segment_tokens=seg)
    for _ in range(3):
        o2, s2 = run(d, segment_tokens=seg)
        assert torch.equal(o, o2) and torch.equal(s, s2)


def test_other_stream():
    import torch

    d = inputs(2, 300, 3, 1, 128, 128, "bf16", "fp32", "g", seed=16)
    o, s = run(d, segment_tokens=64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        o2, s2 = run(d, segment_tokens=64, stream=stream)
        assert torch.equal(o, o2) and torch.equal(s, s2)


@pytest.mark.parametrize("T,seg,lens", [(4, 0, None), (200, -1, None), (200, 64, None),
                                        (200, 64, [150, 0, 50])])
def test_graph(T, seg, lens):
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    d = inputs(1 if lens else 2, T, 3, 1, 128, 128, "bf16", "fp32", "g", seed=17, lens=lens)
    ref_o, ref_s = run(d, segment_tokens=seg)
    a = dict(d)
    q, k, v, g = (a.pop(n) for n in "qkvg")
    o, s = torch.empty_like(ref_o), torch.empty_like(ref_s)
    call = lambda: kda.kda_linear(q, k, v, g, o=o, state_out=s, segment_tokens=seg, **a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        o.zero_()
        s.zero_()
        run(d, segment_tokens=seg)  # eager work between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ref_o) and torch.equal(s, ref_s)


def test_steps_continue_a_prompt():
    """A prompt, then tokens one and three at a time, against the whole."""
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    d = inputs(2, 100, 2, 1, 128, 128, "bf16", "fp32", "g", seed=18)
    ref = oracle(d)
    cut = lambda a, b: [d[n][:, a:b] for n in "qkv"] + [d["g"][:, a:b].contiguous()]
    o, st = kda.kda_linear(*cut(0, 90), d["state_in"])
    outs = [o]
    at = 90
    for n in (1, 1, 3, 3, 1, 1):
        o, _ = kda.kda_linear(*cut(at, at + n), st, state_out=st)
        outs.append(o)
        at += n
    check(torch.cat(outs, 1), st, ref, d, "steps")
