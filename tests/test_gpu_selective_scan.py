"""The selective state space scan (kda_selective_scan) against its recurrence in FP64.

Tolerance, element by element: the oracle carries a bound on the error of FP32 arithmetic along
with the recurrence (see there); a BF16 result adds its rounding, 2^-8 of its value, an FP32
one 2^-24.
"""

import numpy as np
import pytest

from oracle import selective_scan_fp64

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import chunkwise_delta_rule_kda_amd as kda

    kda.load_library()


def dtype(name):
    import torch

    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def host(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def inputs(B, T, D, S=16, G=1, io="bf16", st="fp32", z=True, skip=True, softplus=True, lens=None,
           seed=0, state=True, steps=(1e-3, 1.0), pad=0):
    """Device tensors; steps: range of the channels' typical step sizes; pad: elements between
    the rows of each strided input."""
    import torch

    gen = torch.Generator(device="cuda")
    gen.manual_seed(900 + seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    dt = dtype(io)
    wide = lambda n: r(B, T, n + pad).to(dt)[..., :n]
    step = steps[0] * (steps[1] / steps[0]) ** torch.rand(D, generator=gen, device="cuda")
    d = dict(u=wide(D), A=-torch.rand(D, S, generator=gen, device="cuda") * S - 0.1,
             B=wide(G * S).unflatten(-1, (G, S)), C=wide(G * S).unflatten(-1, (G, S)),
             D=r(D) if skip else None, z=wide(D) if z else None, cu_seqlens=None, state_in=None,
             state_dtype=dt if st == io else dtype(st), delta_softplus=softplus)
    if softplus:
        d["delta"], d["delta_bias"] = wide(D), torch.log(torch.expm1(step))
    else:
        d["delta"], d["delta_bias"] = (step * torch.exp(r(B, T, D))).to(dt), None
    if G == 1:  # the form without an axis of groups
        d["B"], d["C"] = d["B"][:, :, 0], d["C"][:, :, 0]
    N = B
    if lens is not None:
        d["cu_seqlens"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device="cuda",
                                       dtype=torch.int64)
        N = len(lens)
    if state:
        d["state_in"] = r(N, D, S).to(dtype(st))
    return d


def run(d, **kw):
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    d = {**d, **kw}
    first = [d.pop(n) for n in ("u", "delta", "A", "B", "C")]
    out = kda.kda_selective_scan(*first, **d)
    torch.cuda.synchronize()
    return out


def oracle(d, state0=None, segment=0):
    four = lambda x: x if x.ndim == 4 else x[:, :, None]
    cu = None if d["cu_seqlens"] is None else d["cu_seqlens"].cpu().numpy()
    return selective_scan_fp64(host(d["u"]), host(d["delta"]), host(d["A"]), four(host(d["B"])),
                               four(host(d["C"])), host(d["D"]), host(d["z"]),
                               host(d["state_in"]) if state0 is None else state0,
                               delta_bias=host(d["delta_bias"]), softplus=d["delta_softplus"],
                               cu_seqlens=cu, segment=segment)


def within(got, ref, err, name):
    import torch

    u = 2.0 ** -8 if got.dtype == torch.bfloat16 else E
    got, slack = host(got), u * np.abs(ref) + E * err
    assert got.shape == ref.shape and np.all(np.isfinite(got)), name
    if got.size:
        worst = np.max(np.abs(got - ref) / np.maximum(slack, 1e-300))
        print(f"[case] {name}: {worst:.3f} of its bound", flush=True)
        assert worst <= 1, name


def check(d, name, **kw):
    y, s = run(d, **kw)
    y_ref, s_ref, y_err, s_err = oracle(d, segment=max(0, kw.get("segment_tokens", 0)))
    within(y, y_ref, y_err, name + " out")
    within(s, s_ref, s_err, name + " state")
    return y, s


CASES = [
    # B, T, D, S, G, io, st, z, skip, softplus
    (1, 1, 8, 16, 1, "bf16", "fp32", True, True, True),
    (3, 1, 1536, 16, 1, "bf16", "bf16", True, True, True),
    (2, 1, 40, 8, 1, "fp32", "fp32", False, True, False),
    (2, 8, 200, 16, 1, "bf16", "fp32", True, False, True),
    (1, 5, 128, 64, 2, "bf16", "fp32", True, True, True),
    (2, 3, 136, 32, 1, "fp32", "bf16", True, True, True),
    (1, 9, 8, 16, 1, "bf16", "fp32", True, True, True),     # past the token form
    (2, 31, 72, 8, 1, "bf16", "bf16", True, True, False),
    (1, 32, 32, 16, 1, "bf16", "fp32", False, False, True),
    (2, 33, 264, 16, 1, "fp32", "fp32", True, True, True),
    (1, 64, 192, 32, 3, "bf16", "fp32", True, True, True),  # three groups of 64 channels
    (1, 65, 64, 64, 2, "bf16", "bf16", False, True, True),  # two groups of 32
    (3, 100, 40, 64, 1, "fp32", "fp32", True, True, True),
    (1, 257, 104, 16, 1, "bf16", "fp32", True, True, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_the_recurrence(case):
    B, T, D, S, G, io, st, z, skip, softplus = case
    d = inputs(B, T, D, S, G, io, st, z, skip, softplus)
    check(d, f"scan {case}")
    check(dict(d, state_in=None), f"scan {case} from zeros")
    if T <= 8:  # the same tokens by the kernel for prompts
        check(d, f"scan {case} serial", segment_tokens=-1)


@pytest.mark.parametrize("S,io,st", [(16, "bf16", "fp32"), (8, "fp32", "fp32"),
                                     (32, "bf16", "bf16"), (64, "fp32", "fp32")])
@pytest.mark.parametrize("T,seg", [(64, 64), (65, 64), (200, 64), (300, 128), (257, 192)])
def test_segments(T, seg, S, io, st):
    d = inputs(2, T, 72, S, 1, io, st, steps=(1e-3, 0.1))
    check(d, f"scan T={T} segments of {seg}", segment_tokens=seg)
    check(dict(d, state_in=None), f"scan T={T} segments of {seg} from zeros", segment_tokens=seg)


@pytest.mark.parametrize("lens", [[1], [0, 70, 0], [1, 2, 3, 4, 5], [64, 128, 63, 65], [0, 0],
                                  [3] * 70, [200, 1, 0, 40, 7, 64]], ids=str)
@pytest.mark.parametrize("seg", [-1, 64, 128])
def test_packed(lens, seg):
    d = inputs(1, sum(lens), 72, lens=lens, steps=(1e-3, 0.1))
    check(d, f"scan packed {lens} seg={seg}", segment_tokens=seg)
    check(dict(d, state_in=None), f"scan packed {lens} seg={seg} zeros", segment_tokens=seg)


@pytest.mark.parametrize("T", [1, 4, 8, 40])
def test_strides(T):
    import torch

    check(inputs(2, T, 72, pad=24), "scan slices")
    check(inputs(2, T, 128, 16, 2, pad=8), "scan slices of groups")
    d = inputs(1, T, 72, state=False)
    many = lambda t: t.expand(3, *t.shape[1:])
    check(dict(d, **{n: many(d[n]) for n in ("u", "delta", "B", "C", "z")}), "scan expanded")
    d = inputs(5, T, 64)
    for n in ("u", "delta", "B", "C", "z"):  # sequence first
        d[n] = d[n].transpose(0, 1).contiguous().transpose(0, 1)
    check(d, "scan sequence first")


def test_token_calls_continue_a_prompt():
    """A prompt, then one token after another, then three at once, in place: the sequence."""
    import torch

    d = inputs(2, 100, 136, st="fp32")
    y_ref, s_ref, y_err, s_err = oracle(d)
    state, outs = d["state_in"].clone(), []
    cuts = [0, 90, 91, 92, 95, 100]
    for a, b in zip(cuts, cuts[1:]):
        part = {n: d[n][:, a:b] for n in ("u", "delta", "B", "C", "z")}
        y, s = run(dict(d, **part, state_in=state), state_out=state)
        assert s is state
        outs.append(y)
    within(torch.cat(outs, 1), y_ref, y_err, "scan in pieces out")
    within(state, s_ref, s_err, "scan in pieces state")


@pytest.mark.parametrize("T,lens,seg", [(1, None, 0), (6, None, 0), (40, None, -1),
                                        (150, None, 64), (150, [70, 0, 80], 64)])
def test_pool(T, lens, seg):
    """Reads and writes other slots, one slot read by two sequences, ids outside the pool; the
    other slots and the padding between slots stay. Then the same in place."""
    import torch

    N, D, S = 3, 72, 16
    d = inputs(1 if lens else N, T, D, S, lens=lens, steps=(1e-3, 0.1))
    wide = torch.randn(9, D * S + 24, device="cuda")
    pool = wide[:, :D * S].unflatten(1, (D, S))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    start = pool[[4, 4, 0]].clone()
    start[2] = 0  # id -1
    want = wide.clone()
    seg_of = max(0, seg)
    y_ref, s_ref, y_err, s_err = oracle(d, host(start), seg_of)
    d.pop("state_in")
    y, s = run(d, state_in=pool, ssm_state_indices=i32([4, 4, -1]),
               state_out_indices=i32([7, 9, 1]), segment_tokens=seg)
    within(y, y_ref, y_err, f"scan pool T={T}")
    within(pool[[7, 1]], s_ref[[0, 2]], s_err[[0, 2]], f"scan pool T={T} states")
    assert s.data_ptr() == pool.data_ptr()
    for slot in (7, 1):
        want[slot, :D * S] = wide[slot, :D * S]
    assert torch.equal(wide, want)
    y_ref, s_ref, y_err, s_err = oracle(d, host(pool[[7, 3, 1]]), seg_of)
    y, _ = run(d, state_in=pool, ssm_state_indices=i32([7, 3, 1]), segment_tokens=seg)
    within(y, y_ref, y_err, f"scan pool in place T={T}")
    within(pool[[7, 3, 1]], s_ref, s_err, f"scan pool in place T={T} states")
    for slot in (7, 3, 1):
        want[slot, :D * S] = wide[slot, :D * S]
    assert torch.equal(wide, want)


def test_no_state_written_and_empty_calls():
    import torch

    for seg in (0, -1, 64):
        d = inputs(2, 150, 72)
        kept = d["state_in"].clone()
        y, s = run(d, segment_tokens=seg)
        y2, s2 = run(d, output_final_state=False, segment_tokens=seg)
        assert s2 is None and torch.equal(y, y2) and torch.equal(d["state_in"], kept)
    d = inputs(2, 0, 72)
    y, s = run(d)
    assert y.shape == (2, 0, 72) and torch.equal(s, d["state_in"])


def test_extreme_steps():
    """Step sizes from nothing to where the state is gone at once: exact at both ends."""
    import torch

    d = inputs(1, 40, 64, io="fp32", skip=False, z=False)
    d["delta"][:, ::3] = -60.0   # e^-60: the state stays
    d["delta"][:, 1::3] = 90.0   # exp(90 A) A <= -0.1 ...
    d["A"] = d["A"] - 2.0        # ... is below 2^-126
    check(d, "scan extreme steps")
    check(d, "scan extreme steps, segments", segment_tokens=64)


def test_infinities_stay_in_their_channel():
    import torch

    for T, seg in ((6, 0), (150, -1), (150, 64)):
        d = inputs(2, T, 72)
        bad = dict(d, u=d["u"].clone())
        bad["u"][0, 3, 5] = float("inf")
        y, s = run(d, segment_tokens=seg)
        y2, s2 = run(bad, segment_tokens=seg)
        touched = torch.zeros(y.shape, dtype=torch.bool, device="cuda")
        touched[0, 3:, 5] = True
        assert torch.equal(y[~touched], y2[~touched]) and not torch.isfinite(y2[0, 3, 5])
        s2[0, 5] = s[0, 5]
        assert torch.equal(s, s2)


@pytest.mark.parametrize("T,seg", [(3, 0), (100, -1), (300, 64)])
def test_other_stream_graph_and_repeat(T, seg):
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    d = inputs(3, T, 136)
    y, s = run(d, segment_tokens=seg)
    y1, s1 = run(d, segment_tokens=seg)
    assert torch.equal(y, y1) and torch.equal(s, s1)  # bit by bit
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, s2 = run(d, stream=side, segment_tokens=seg)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(s, s2)

    out, end = torch.empty_like(y), torch.empty_like(s)
    call = lambda: kda.kda_selective_scan(
        d["u"], d["delta"], d["A"], d["B"], d["C"], d["D"], d["z"], d["state_in"],
        delta_bias=d["delta_bias"], out=out, state_out=end, segment_tokens=seg)
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        d["u"].copy_(torch.randn_like(d["u"]))
        want, want_end = run(d, segment_tokens=seg)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(end, want_end)


@pytest.mark.parametrize("B,D,S,G,io,st", [
    (70, 1928, 16, 1, "bf16", "fp32"),   # the last wave's channels partly behind the end
    (70, 1920, 16, 30, "bf16", "bf16"),  # a row of B and C for each wave of 64 channels
    (66, 2016, 16, 63, "fp32", "fp32"),  # for each 32 channels: less than a wave has
    (70, 1928, 8, 1, "bf16", "fp32"),
    (70, 1000, 32, 1, "fp32", "bf16"),
    (35, 968, 64, 1, "bf16", "fp32"),
])
@pytest.mark.parametrize("T", [1, 3])
def test_many_tokens(B, D, S, G, io, st, T):
    """Calls large enough for several channels in a lane of the token form."""
    check(inputs(B, T, D, S, G, io, st), f"scan {B} x {T} tokens, {D} channels, {S} states")


def test_rows_behind_the_last_sequence_stay():
    import torch

    for seg in (-1, 64):
        d = inputs(1, 150, 72, lens=[70, 0, 50], steps=(1e-3, 0.1))
        out = torch.full((1, 150, 72), 7.0, device="cuda", dtype=torch.bfloat16)
        y, s = run(d, out=out, segment_tokens=seg)
        assert bool((y[:, 120:] == 7).all())
        first = {n: d[n][:, :120] for n in ("u", "delta", "B", "C", "z")}
        y2, s2 = run(dict(d, **first), segment_tokens=seg)
        assert torch.equal(y[:, :120], y2) and torch.equal(s, s2)


def test_two_streams_at_once():
    import torch

    d = [inputs(2, 600, 136, seed=i) for i in range(2)]
    want = [run(x, segment_tokens=64) for x in d]
    streams = [torch.cuda.Stream() for _ in d]
    torch.cuda.synchronize()
    import chunkwise_delta_rule_kda_amd as kda

    got = []
    for _ in range(4):
        for x, s in zip(d, streams):
            a = dict(x, stream=s, segment_tokens=64)
            first = [a.pop(n) for n in ("u", "delta", "A", "B", "C")]
            got.append(kda.kda_selective_scan(*first, **a))
    torch.cuda.synchronize()
    for i, (y, s) in enumerate(got):
        assert torch.equal(y, want[i % 2][0]) and torch.equal(s, want[i % 2][1])


def test_automatic_geometry_of_long_prompts():
    """The segments that the library takes by itself, against the oracle."""
    import chunkwise_delta_rule_kda_amd as kda

    for lens in (None, [3000, 1, 1096]):
        d = inputs(1, 4097, 40, lens=lens, steps=(1e-3, 0.1), io="fp32")
        N = 1 if lens is None else 3
        plan = kda.kda_selective_scan_plan(kda.make_selective_scan_args(
            B=1, T=4097, D=40, N=N, io_dtype=1, state_dtype=1, flags=1,
            cu_seqlens=None if lens is None else d["cu_seqlens"]))
        assert plan["segment_tokens"] > 0
        y, s = run(d)
        y_ref, s_ref, y_err, s_err = oracle(d, segment=plan["segment_tokens"])
        within(y, y_ref, y_err, f"scan 4097 tokens {lens} out")
        within(s, s_ref, s_err, f"scan 4097 tokens {lens} state")
