"""kda_selective_scan in the geometries that its own tests leave out: several groups of B and C
with segments and packed batches, more than two blocks of 32 channels with segments, step sizes
at both ends carried over segments, packed batches about the bound up to which the longest
sequence runs first, one long sequence among many short ones, offsets past 2^32, calls without
tokens in pools, very many sequences, and captured packed calls whose lengths change. Every
case that means segments asserts them on the plan.

Tolerance: as in test_gpu_selective_scan.py, the oracle's bound on FP32 arithmetic and the
result's own rounding, element by element."""

import numpy as np
import pytest

from test_gpu_selective_scan import _gpu, check, dtype, inputs, oracle, run, within  # noqa: F401

pytestmark = pytest.mark.gpu


def plan(d, segment_tokens=0):
    import chunkwise_delta_rule_kda_amd as kda

    B, T, D = d["u"].shape
    cu = d["cu_seqlens"]
    code = {dtype("bf16"): 0, dtype("fp32"): 1}
    return kda.kda_selective_scan_plan(kda.make_selective_scan_args(
        B=B, T=T, D=D, S=d["A"].shape[1], G=d["B"].shape[2] if d["B"].dim() == 4 else 1,
        N=B if cu is None else cu.numel() - 1, io_dtype=code[d["u"].dtype],
        state_dtype=code[d["state_dtype"]], flags=int(d["delta_softplus"]), cu_seqlens=cu,
        state_in=d["state_in"], segment_tokens=segment_tokens))


def segmented(d, name, seg, **kw):
    assert plan(d, seg)["segment_tokens"] == seg
    return check(d, name, segment_tokens=seg, **kw)


@pytest.mark.parametrize("D,S,G,io,st", [
    (288, 16, 3, "bf16", "fp32"),  # groups of 96 channels: three blocks each
    (64, 32, 2, "fp32", "fp32"),   # of one block
    (160, 8, 5, "bf16", "bf16"),
    (192, 64, 2, "fp32", "bf16"),
])
@pytest.mark.parametrize("lens", [None, [200, 1, 0, 40, 7, 64, 130]], ids=["fixed", "packed"])
def test_groups_with_segments(D, S, G, io, st, lens):
    d = inputs(1 if lens else 2, sum(lens) if lens else 200, D, S, G, io, st, lens=lens,
               steps=(1e-3, 0.1), pad=8)
    for seg in (64, 128):
        segmented(d, f"scan {G} groups of {D // G}, segments of {seg}", seg)
        segmented(dict(d, state_in=None), f"scan {G} groups, segments of {seg}, zeros", seg)
    if lens:
        check(d, f"scan {G} groups packed serial", segment_tokens=-1)


@pytest.mark.parametrize("D,S,G,io", [(1032, 16, 1, "bf16"), (520, 64, 1, "fp32"),
                                      (416, 32, 13, "bf16"), (1000, 8, 1, "fp32")])
def test_many_channel_blocks_with_segments(D, S, G, io):
    d = inputs(2, 150, D, S, G, io, steps=(1e-3, 0.1))
    segmented(d, f"scan {D} channels, segments", 64)
    d = inputs(1, 170, D, S, G, io, lens=[66, 0, 104], steps=(1e-3, 0.1), seed=1)
    segmented(d, f"scan {D} channels packed, segments", 64)


@pytest.mark.parametrize("S,io,st", [(16, "fp32", "fp32"), (32, "fp32", "bf16"),
                                     (8, "bf16", "fp32"), (64, "fp32", "fp32")])
@pytest.mark.parametrize("lens", [None, [130, 0, 70]], ids=["fixed", "packed"])
def test_extreme_steps_over_segments(S, io, st, lens):
    """The sums of a segment's step sizes where they vanish and where exp(sum A) does: channels
    that keep their state to the end, that lose it at every token, and ordinary ones."""
    d = inputs(1, 200, 64, S, io=io, st=st, skip=False, z=False, lens=lens)
    d["delta_bias"] = None
    d["delta"] = d["delta"].clone()
    d["delta"][..., ::3] = -60.0  # e^-60
    d["delta"][..., 1::3] = 90.0
    d["A"] = d["A"] - 2.0         # exp(90 A) is below 2^-126
    segmented(d, "scan extreme steps, segments", 64)
    # and steps of exactly nothing: the state passes all segments as it is
    d["delta_softplus"] = False
    d["delta"] = d["delta"] * 0
    _, s = segmented(d, "scan steps of nothing, segments", 64)
    import torch

    assert torch.equal(s, d["state_in"])


@pytest.mark.parametrize("N", [2, 63, 64, 65])
def test_packed_about_the_bound_of_the_order_by_length(N):
    """Up to 64 sequences the longest ones run first: with ties, empty ones and every place of
    the longest."""
    for turn in (0, N // 2, N - 1):
        lens = [(11 * ((i + turn) % N)) % 37 for i in range(N)]
        lens[turn] = 80
        d = inputs(1, sum(lens), 40, lens=lens, seed=turn)
        assert plan(d, -1)["segment_tokens"] == 0
        check(d, f"scan {N} packed, the longest at {turn}", segment_tokens=-1)
        check(d, f"scan {N} packed, the longest at {turn}, automatic",
              segment_tokens=plan(d)["segment_tokens"] or -1)


@pytest.mark.parametrize("lens", [[1] * 20 + [2000] + [1] * 43, [1500] + [0, 1] * 60], ids=["64", "121"])
def test_one_long_sequence_among_short_ones(lens):
    """A prompt in one packed call with other sequences' tokens: as the library plans it, and cut
    on the caller's word, which is the faster form here."""
    d = inputs(1, sum(lens), 136, lens=lens, steps=(1e-3, 0.1))
    seg = plan(d)["segment_tokens"]
    y, s = run(d)
    y_ref, s_ref, y_err, s_err = oracle(d, segment=seg)
    within(y, y_ref, y_err, f"scan one of {len(lens)} long out")
    within(s, s_ref, s_err, f"scan one of {len(lens)} long state")
    segmented(d, f"scan one of {len(lens)} long, segments", 256)


def test_offsets_past_32_bits():
    """Batch and slot strides past 2^32 bytes, and a packed call of more than 2^31 elements."""
    import torch

    far = (1 << 31) + 64  # elements between sequences and slots
    for T, seg in ((2, 0), (70, -1), (200, 64)):
        d = inputs(2, T, 72, steps=(1e-3, 0.1))
        for n in ("u", "delta", "z", "B", "C"):
            t = d[n]
            wide = torch.empty(far + t[0].numel(), dtype=t.dtype, device="cuda").as_strided(
                t.shape, (far, t.shape[2], 1))
            d[n] = wide.copy_(t)
        pool = torch.empty(2 * far + 72 * 16, device="cuda").as_strided((3, 72, 16), (far, 16, 1))
        pool[0], pool[2] = d["state_in"][0], d["state_in"][1]
        y_ref, s_ref, y_err, s_err = oracle(d, segment=max(0, seg))
        d["state_in"] = pool
        y, _ = run(d, ssm_state_indices=torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
                   segment_tokens=seg)
        within(y, y_ref, y_err, f"scan far apart T={T} out")
        within(pool[[0, 2]], s_ref, s_err, f"scan far apart T={T} state")
        del wide, pool, d
        torch.cuda.empty_cache()


def test_rows_past_31_bits():
    """8200 channels x 262,200 tokens of two sequences. Decays of exp(-200) and less are zero, so
    the last tokens are those of a short call, bit by bit."""
    import torch

    D, T = 8200, 262200
    d = inputs(1, 64, D, z=False, softplus=False, state=False)
    d["A"] = -200 - torch.rand_like(d["A"])
    rows = dict(u=d["u"], delta=torch.ones_like(d["delta"][:, :1]).expand(1, 64, D), B=d["B"],
                C=d["C"])
    want, end = run(dict(d, **rows), segment_tokens=-1)
    long = {n: torch.zeros(1, T, t.shape[2], dtype=t.dtype, device="cuda")
            for n, t in rows.items() if n != "delta"}
    for n, t in long.items():
        t[:, -64:] = rows[n]
        t[:, :64] = rows[n]
    long["delta"] = torch.ones_like(d["delta"][:, :1]).expand(1, T, D)
    cu = torch.tensor([0, 1000, T], device="cuda")
    for seg in (-1, 65536):
        y, s = run(dict(d, **long, cu_seqlens=cu), segment_tokens=seg)
        assert torch.equal(y[:, -64:], want) and torch.equal(y[:, :64], want)
        assert torch.equal(s[1:], end) and not y[:, 64:-64].any()
        del y, s


def test_state_types_of_calls_without_a_state():
    """state_dtype as documented: the inputs' type unless asked for. And what the documentation
    warns of: carried in BF16 under decays closer to 1 than 2^-9 a state stands still (half a
    unit of its last place is at least 2^-9 of it), in FP32 it follows the recurrence."""
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    d = inputs(2, 1, 72, state=False, softplus=False)
    call = lambda state, **kw: kda.kda_selective_scan(
        d["u"], d["delta"], d["A"], d["B"], d["C"], d["D"], d["z"], state, delta_softplus=False, **kw)[1]
    assert call(None).dtype == torch.bfloat16
    assert call(None, state_dtype=torch.float32).dtype == torch.float32
    x, w = d["u"], torch.ones(72, 4, device="cuda")
    assert kda.kda_short_conv(x, w)[1].dtype == torch.bfloat16
    assert kda.kda_short_conv(x, w, state_dtype=torch.float32)[1].dtype == torch.float32
    d["u"], d["delta"], d["A"] = d["u"] * 0, d["delta"] * 0 + 1, d["A"] * 0 - 2.0 ** -10
    first = torch.randn(2, 72, 16, device="cuda").bfloat16()
    few, full = first, first.float()
    for _ in range(200):
        few, full = call(few), call(full)
    assert torch.equal(few, first)
    want = first.double() * torch.exp(torch.tensor(-200 * 2.0 ** -10, dtype=torch.float64))
    # a token's exponential is off by 3 units of 2^-24 at most, its product by one
    assert bool(((full.double() - want).abs() <= 200 * 4 * 2.0 ** -24 * want.abs()).all())


@pytest.mark.parametrize("S", [8, 32])
def test_no_tokens_in_a_pool(S):
    import torch

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ids = dict(ssm_state_indices=i32([2, 2, 9]), state_out_indices=i32([6, 0, 4]))
    for lens in (None, [0, 0, 0]):
        d = inputs(1 if lens else 3, 0, 72, S, lens=lens, state=False)
        pool = torch.randn(7, 72, S, device="cuda")
        want = pool.clone()
        want[[6, 0]] = pool[[2, 2]]
        want[4] = 0
        run(dict(d, state_in=pool), **ids)
        assert torch.equal(pool, want)


def test_very_many_sequences():
    import torch

    d = inputs(70001, 1, 8)
    y, s = run(d)
    pick = [0, 1, 4095, 4096, 65535, 65536, 70000]
    part = dict(d, **{n: d[n][pick] for n in ("u", "delta", "B", "C", "z", "state_in")})
    y_ref, s_ref, y_err, s_err = oracle(part)
    within(y[pick], y_ref, y_err, "scan 70001 tokens out")
    within(s[pick], s_ref, s_err, "scan 70001 tokens state")
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(s).all())
    lens = [int(n) for n in np.random.default_rng(2).integers(0, 4, 5000)]
    lens[4321] = 200
    d = inputs(1, sum(lens), 8, lens=lens)
    check(d, "scan packed 5000 sequences", segment_tokens=-1)
    segmented(d, "scan packed 5000 sequences, segments", 64)


@pytest.mark.parametrize("seg", [-1, 64])
def test_captured_packed_call_with_other_lengths(seg):
    """The lengths are read on the device: a captured call follows them, cut or not."""
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    d = inputs(1, 250, 72, lens=[70, 0, 180])
    out, end = torch.empty_like(d["u"]), torch.empty_like(d["state_in"])
    call = lambda: kda.kda_selective_scan(
        d["u"], d["delta"], d["A"], d["B"], d["C"], d["D"], d["z"], d["state_in"], d["cu_seqlens"],
        delta_bias=d["delta_bias"], out=out, state_out=end, segment_tokens=seg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for cu in ([0, 0, 249, 250], [0, 250, 250, 250], [0, 63, 128, 250]):
        d["cu_seqlens"].copy_(torch.tensor(cu))
        d["u"].copy_(torch.randn_like(d["u"]))
        want, want_end = run(d, segment_tokens=seg)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(end, want_end)
