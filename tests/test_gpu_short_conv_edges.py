"""kda_short_conv at its edges: offsets past 32 bits, calls without tokens, very many sequences,
and captured packed calls whose lengths change. Tolerances as in test_gpu_short_conv.py."""

import numpy as np
import pytest

from test_gpu_short_conv import _gpu, check, check_out, host, inputs, oracle, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 50])
def test_sequences_and_slots_far_apart(T):
    import torch

    far, C, W = (1 << 31) + 64, 136, 4
    d = inputs(2, T, C, W)
    x, state = d["x"], d["state_in"]
    y_ref, s_ref, err = oracle(d)
    d["x"] = torch.empty(far + x[0].numel(), dtype=x.dtype, device="cuda").as_strided(
        x.shape, (far, C, 1)).copy_(x)
    pool = torch.empty(2 * far + state[0].numel(), dtype=state.dtype, device="cuda").as_strided(
        (3, W - 1, C), (far, C, 1))
    pool[0], pool[2] = state[0], state[1]
    d["state_in"] = pool
    ids = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    y, _ = run(d, ssm_state_indices=ids)
    check_out(y, y_ref, err, f"conv far apart T={T}")
    assert np.array_equal(host(pool[[0, 2]]), s_ref)


def test_rows_past_31_bits():
    """60,000 tokens x 36864 channels of three sequences: windows across the whole range are those
    of short calls from the rows before them, bit by bit."""
    import torch

    T, C = 60000, 36864
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.randn(1, T, C, generator=gen, device="cuda", dtype=torch.bfloat16)
    d = inputs(1, 1, C, state=False)
    cu = torch.tensor([0, 100, 101, T], device="cuda")
    y, s = run(dict(d, x=x, cu_seqlens=cu))
    for a, b in ((0, 100), (100, 101), (101, 130)):
        part, _ = run(dict(d, x=x[:, a:b]))
        assert torch.equal(part, y[:, a:b])
    for a in (30000, 58254, 58255, T - 40):  # 58254 x 36864 is the last row begun below 2^31
        part, _ = run(dict(d, x=x[:, a:a + 40]), state_in=x[:, a - 3:a].contiguous())
        assert torch.equal(part, y[:, a:a + 40])
    assert torch.equal(s[0], x[0, 97:100]) and torch.equal(s[2], x[0, T - 3:])
    assert torch.equal(s[1, 2], x[0, 100]) and not s[1, :2].any()


@pytest.mark.parametrize("io,st,W", [("bf16", "fp32", 4), ("fp32", "bf16", 2)])
def test_no_tokens(io, st, W):
    """States pass a call of no tokens: dense, in place, and from slot to slot of a pool."""
    import torch

    d = inputs(3, 0, 72, W, io, st)
    y, s = run(d)
    assert y.shape == (3, 0, 72) and torch.equal(s, d["state_in"])
    kept = d["state_in"].clone()
    _, s = run(d, state_out=d["state_in"])
    assert torch.equal(s, kept) and not run(dict(d, state_in=None))[1].any()
    pool = torch.randn(7, W - 1, 72, device="cuda").to(kept.dtype)
    want = pool.clone()
    want[[6, 0]] = pool[[2, 2]]
    want[4] = 0
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    run(d, state_in=pool, ssm_state_indices=i32([2, 2, 9]), state_out_indices=i32([6, 0, 4]))
    assert torch.equal(pool, want)


@pytest.mark.parametrize("C", [8, 40])
def test_very_many_sequences(C):
    import torch

    d = inputs(70001, 1, C)
    y, s = run(d)
    pick = [0, 1, 4095, 4096, 65535, 65536, 70000]
    part = dict(d, x=d["x"][pick], state_in=d["state_in"][pick])
    y_ref, s_ref, err = oracle(part)
    check_out(y[pick], y_ref, err, "conv 70001 tokens")
    assert np.array_equal(host(s[pick]), s_ref) and bool(torch.isfinite(y).all())
    rng = np.random.default_rng(C)
    lens = [int(n) for n in rng.integers(0, 4, 5000)]  # 64 candidates at a time, three times
    check(inputs(1, sum(lens), C, lens=lens), f"conv packed 5000 sequences, {C} channels")


def test_captured_packed_call_with_other_lengths():
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    d = inputs(1, 150, 136, lens=[70, 0, 80])
    out, end = torch.empty_like(d["x"]), torch.empty_like(d["state_in"])
    call = lambda: kda.kda_short_conv(d["x"], d["weight"], d["bias"], d["state_in"],
                                      d["cu_seqlens"], out=out, state_out=end)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for cu in ([0, 0, 149, 150], [0, 150, 150, 150], [0, 15, 32, 150]):
        d["cu_seqlens"].copy_(torch.tensor(cu))
        d["x"].copy_(torch.randn_like(d["x"]))
        want, want_end = run(d)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(end, want_end)
