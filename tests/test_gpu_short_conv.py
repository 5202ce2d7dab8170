"""The short causal convolution (kda_short_conv) against its definition in FP64.

Tolerance, element by element: the oracle's bound on the FP32 arithmetic plus the result's own
rounding (2^-8 of a BF16 value, 2^-24 of an FP32 one). The final state holds inputs, so it is
compared bit by bit (an FP32 input in a BF16 state with its rounding to nearest even).
"""

import numpy as np
import pytest

from oracle import short_conv_fp64

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


def inputs(B, T, C, W=4, io="bf16", st="bf16", bias=True, lens=None, seed=0, state=True,
           stride=None):
    """Device tensors; stride: the token stride where x is a part of wider rows."""
    import torch

    gen = torch.Generator(device="cuda")
    gen.manual_seed(500 + seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    d = dict(x=r(B, T, stride or C).to(dtype(io))[..., :C], weight=r(C, W) * W ** -0.5,
             bias=0.1 * r(C) if bias else None, cu_seqlens=None, state_in=None,
             state_dtype=dtype(st))
    N = B
    if lens is not None:
        d["cu_seqlens"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), device="cuda",
                                       dtype=torch.int64)
        N = len(lens)
    if state:
        d["state_in"] = r(N, W - 1, C).to(dtype(st))
    return d


def run(d, **kw):
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    d = {**d, **kw}
    x, w, b = d.pop("x"), d.pop("weight"), d.pop("bias")
    out = kda.kda_short_conv(x, w, b, **d)
    torch.cuda.synchronize()
    return out


def oracle(d, state0=None, silu=True):
    cu = None if d["cu_seqlens"] is None else d["cu_seqlens"].cpu().numpy()
    return short_conv_fp64(host(d["x"]), host(d["weight"]), host(d["bias"]),
                           host(d["state_in"]) if state0 is None else state0, cu_seqlens=cu,
                           silu=silu)


def check_out(y, ref, err, name):
    import torch

    u = 2.0 ** -8 if y.dtype == torch.bfloat16 else E
    got, slack = host(y), u * np.abs(ref) + E * err
    assert got.shape == ref.shape and np.all(np.isfinite(got)), name
    if got.size:
        worst = np.max(np.abs(got - ref) / np.maximum(slack, 1e-300))
        print(f"[case] {name}: {worst:.3f} of its bound", flush=True)
        assert worst <= 1, name


def check(d, name, silu=True, **kw):
    import torch

    y, s = run(d, activation="silu" if silu else None, **kw)
    y_ref, s_ref, err = oracle(d, silu=silu)
    check_out(y, y_ref, err, name)
    assert torch.equal(s.cpu(), torch.from_numpy(s_ref).float().to(s.dtype)), name
    return y, s


CASES = [
    # B, T, C, W, io, st, bias
    (1, 1, 8, 4, "bf16", "bf16", False),      # one token of the narrowest row
    (3, 1, 2304, 4, "bf16", "fp32", True),
    (2, 2, 264, 4, "bf16", "bf16", True),     # shorter than the window
    (1, 3, 72, 4, "fp32", "fp32", True),      # exactly the window's rows before
    (2, 4, 520, 3, "fp32", "bf16", False),
    (5, 8, 128, 2, "bf16", "bf16", True),
    (1, 17, 2312, 4, "bf16", "fp32", True),   # a run and one token
    (2, 31, 768, 3, "bf16", "bf16", False),
    (1, 33, 40, 2, "fp32", "fp32", True),
    (2, 129, 1032, 4, "bf16", "bf16", True),
    (1, 700, 264, 4, "bf16", "fp32", True),
]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_the_definition(case, silu):
    B, T, C, W, io, st, bias = case
    check(inputs(B, T, C, W, io, st, bias), f"conv {case} silu={silu}", silu)
    check(inputs(B, T, C, W, io, st, bias, state=False, seed=1), f"conv {case} from zeros", silu)


@pytest.mark.parametrize("lens", [[1], [0, 5, 0], [1, 2, 3, 4, 5], [16, 16, 17, 15], [0, 0, 0],
                                  [3] * 90, [200, 1, 0, 40, 7, 64]], ids=str)
@pytest.mark.parametrize("C,W,io", [(40, 4, "bf16"), (520, 3, "fp32"), (8, 2, "bf16")])
def test_packed(lens, C, W, io):
    d = inputs(1, sum(lens), C, W, io, io, lens=lens)
    check(d, f"conv packed {lens} C={C}")
    check(dict(d, state_in=None), f"conv packed {lens} C={C} from zeros")


def test_one_window_over_two_calls():
    """A sequence in pieces, each from the state the piece before left, is the sequence."""
    import torch

    for io in ("bf16", "fp32"):
        d = inputs(2, 23, 136, 4, io, io)
        whole, end = run(d)
        cuts, state, parts = [0, 1, 3, 5, 16, 23], d["state_in"], []
        for a, b in zip(cuts, cuts[1:]):
            y, state = run(dict(d, x=d["x"][:, a:b], state_in=state))
            parts.append(y)
        assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(state, end)


def test_strided_rows_and_expanded_batch():
    d = inputs(2, 40, 264, io="bf16", stride=264 * 3 + 8)
    check(d, "conv slice of a projection")
    d = inputs(1, 40, 264, io="fp32")
    check(dict(d, x=d["x"].expand(3, 40, 264), state_in=None), "conv one row for a batch")
    d = inputs(5, 1, 64)
    d["x"] = d["x"].transpose(0, 1).contiguous().transpose(0, 1)  # sequence-first tokens
    check(d, "conv sequence-first tokens")


def test_in_place_state_and_none():
    import torch

    for T in (1, 2, 40):
        d = inputs(3, T, 264)
        y, s = run(d)
        kept = d["state_in"].clone()
        y2, s2 = run(d, state_out=d["state_in"])
        assert s2 is d["state_in"] and torch.equal(s2, s) and torch.equal(y2, y)
        d["state_in"] = kept
        y3, s3 = run(d, output_final_state=False)
        assert s3 is None and torch.equal(y3, y) and torch.equal(d["state_in"], kept)


@pytest.mark.parametrize("T,lens", [(1, None), (5, None), (30, [12, 0, 18])])
def test_pool(T, lens):
    """Reads and writes other slots, one slot read by two sequences, ids outside the pool; the
    other slots and the padding between slots stay."""
    import torch

    N, C, W = 3, 136, 4
    d = inputs(1 if lens else N, T, C, W, lens=lens)
    wide = torch.randn(9, (W - 1) * C + 24, device="cuda").bfloat16()
    pool = wide[:, :(W - 1) * C].unflatten(1, (W - 1, C))
    before = wide.clone()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    start = pool[[4, 4, 0]].clone()
    start[2] = 0  # id -1
    y_ref, s_ref, err = oracle(d, host(start))
    d.pop("state_in")
    y, s = run(d, state_in=pool, ssm_state_indices=i32([4, 4, -1]),
               state_out_indices=i32([7, 9, 1]))
    check_out(y, y_ref, err, f"conv pool T={T}")
    assert s.data_ptr() == pool.data_ptr()
    want = before.clone()
    for n, slot in ((0, 7), (2, 1)):
        want[slot, :(W - 1) * C] = torch.from_numpy(s_ref[n].reshape(-1)).to(wide)
    assert torch.equal(wide, want)
    # and in place
    y, _ = run(d, state_in=pool, ssm_state_indices=i32([7, 3, 1]))
    y_ref, s_ref, err = oracle(d, host(want[[7, 3, 1], :(W - 1) * C].unflatten(1, (W - 1, C))))
    check_out(y, y_ref, err, f"conv pool in place T={T}")
    for n, slot in enumerate((7, 3, 1)):
        want[slot, :(W - 1) * C] = torch.from_numpy(s_ref[n].reshape(-1)).to(wide)
    assert torch.equal(wide, want)


def test_infinities_stay_in_their_windows():
    import torch

    d = inputs(2, 40, 64, 4, state=True)
    d["x"][0, 20, 8] = float("inf")
    d["state_in"][1, 0, 16] = float("nan")
    y, s = run(d)
    clean = dict(d, x=d["x"].clone(), state_in=d["state_in"].clone())
    clean["x"][0, 20, 8] = 0
    clean["state_in"][1, 0, 16] = 0
    ref, _ = run(clean)
    touched = torch.zeros(y.shape, dtype=torch.bool, device="cuda")
    touched[0, 20:24, 8] = True
    touched[1, 0, 16] = True
    assert torch.equal(y[~touched], ref[~touched])
    assert not torch.isfinite(y[1, 0, 16]) and bool(torch.isfinite(s).all())


def test_other_stream_and_graph():
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    d = inputs(3, 50, 264)
    y, s = run(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, s2 = run(d, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(s, s2)

    out, end = torch.empty_like(y), torch.empty_like(s)
    call = lambda: kda.kda_short_conv(d["x"], d["weight"], d["bias"], d["state_in"], out=out,
                                      state_out=end, state_dtype=d["state_dtype"])
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        d["x"].copy_(torch.randn_like(d["x"]))
        want, want_end = run(d)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(end, want_end)


def test_rows_behind_the_last_sequence_stay():
    import torch

    d = inputs(1, 90, 136, lens=[40, 0, 30])
    out = torch.full((1, 90, 136), 7.0, device="cuda", dtype=torch.bfloat16)
    y, s = run(d, out=out)
    assert bool((y[:, 70:] == 7).all())
    y2, s2 = run(dict(d, x=d["x"][:, :70]))
    assert torch.equal(y[:, :70], y2) and torch.equal(s, s2)


def test_large_call():
    """More than 64 million elements: shorter runs of a thread. Sixteen channels of each end and the
    middle against the definition."""
    import torch

    d = inputs(1, 8192, 8200, 4)
    y, s = run(d)
    pick = torch.tensor([*range(16), *range(4096, 4112), *range(8184, 8200)], device="cuda")
    part = dict(d, x=d["x"][..., pick], weight=d["weight"][pick], bias=d["bias"][pick],
                state_in=d["state_in"][..., pick])
    y_ref, s_ref, err = oracle(part)
    check_out(y[..., pick], y_ref, err, "conv 8192 x 8200")
    assert torch.equal(s[..., pick].cpu(), torch.from_numpy(s_ref).float().to(s.dtype))
    # every element at least finite, and each row like that of a short call from its window
    assert bool(torch.isfinite(y).all())
    for t in (7, 8, 4095, 8190):
        state = d["x"][:, t - 3:t].contiguous()
        one, _ = run(dict(d, x=d["x"][:, t:t + 1], state_in=state))
        assert torch.equal(one[:, 0], y[:, t])
