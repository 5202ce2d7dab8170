"""kda_linear in the geometries that the automatic rule takes for large calls: 128 value rows
per workgroup over several chunks and segments, rings that wrap, packed batches and FP32
calls from and into pool slots, and the automatic segments themselves. Every case asserts
the plan it is meant for, so that another fit of the rule cannot drop it unseen.

The tolerances are those of test_gpu_linear.py, derived there: the geometry changes which
partial sums are formed, not how often a term is rounded (a state that crosses a segment
border stays in FP32, its decay and addition are among the eight operations per chunk that
the bound counts). The oracle is the recurrence in FP64, token after token, on the device.
"""

import numpy as np
import pytest

from test_gpu_linear import U, fp32_part, inputs, oracle, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import chunkwise_delta_rule_kda_amd as kda

    kda.load_library()


def exact(d, state0=None):
    """(o, state, o_abs, state_abs) as oracle.linear_recurrence_fp64, on the device."""
    import torch

    f64 = torch.float64
    B, T, Hk, K = d["q"].shape
    H, V = d["v"].shape[2:]
    rep = lambda x: x.to(f64).repeat_interleave(H // Hk, 2)
    q, k, v = rep(d["q"]), rep(d["k"]), d["v"].to(f64)
    ld = torch.zeros(B, T, H, dtype=f64, device=q.device)
    if d["g"] is not None:
        ld += d["g"].to(f64)
    if d["log_decay"] is not None:
        ld += d["log_decay"].to(f64)
    decay = torch.exp(ld)
    if d["cu_seqlens"] is None:
        spans = [(slice(0, B), 0, T)]
        N = B
    else:
        cu = d["cu_seqlens"].tolist()
        spans = [(slice(0, 1), a, b) for a, b in zip(cu[:-1], cu[1:])]
        N = len(spans)
    start = d["state_in"] if state0 is None else state0
    S_all = torch.zeros(N, H, V, K, dtype=f64, device=q.device) if start is None else start.to(f64)
    o, o_abs = torch.zeros_like(v), torch.zeros_like(v)
    ends, ends_abs = [], []
    at = 0
    for rows, lo, hi in spans:
        n = rows.stop - rows.start
        S = S_all[at:at + n].clone()
        A = S.abs()
        at += n
        for t in range(lo, hi):
            w = v[rows, t][..., None] * k[rows, t][:, :, None]
            f = decay[rows, t][..., None, None]
            S = S * f + w
            A = A * f + w.abs()
            o[rows, t] = (S * q[rows, t][:, :, None]).sum(-1) * K ** -0.5
            o_abs[rows, t] = (A * q[rows, t][:, :, None].abs()).sum(-1) * K ** -0.5
        ends.append(S)
        ends_abs.append(A)
    return o, torch.cat(ends), o_abs, torch.cat(ends_abs)


def within(got, ref, slack, name):
    import torch

    assert got.shape == ref.shape and bool(got.isfinite().all()), name
    if not got.numel():
        return
    err = (got.to(torch.float64) - ref).abs()
    worst = float((err / slack.clamp(min=1e-300)).max())
    print(f"[case] {name}: largest error is {worst:.3f} of its bound", flush=True)
    assert bool((err <= slack).all()), (name, worst)


def check(o, s, ref, d, name):
    import torch

    o_ref, s_ref, o_abs, s_abs = ref
    T, K = d["q"].shape[1], d["q"].shape[3]
    e = fp32_part(T, K)
    bf16 = d["q"].dtype == torch.bfloat16
    within(o, o_ref, U * o_ref.abs() + (2 * U + e) * o_abs if bf16 else e * o_abs, name + " o")
    own = U * s_ref.abs() if s.dtype == torch.bfloat16 else 0.0
    term = (U if s.dtype == torch.bfloat16 else 2.0 ** -24) if bf16 else 0.0
    within(s, s_ref, own + (term + e) * s_abs, name + " state")


def plan(d, segment_tokens=0):
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    B, T, Hk, K = d["q"].shape
    H, V = d["v"].shape[2:]
    cu = d["cu_seqlens"]
    code = lambda dt: 0 if dt == torch.bfloat16 else 1
    return kda.kda_linear_plan(kda.make_linear_args(
        B=B, T=T, H=H, Hk=Hk, K=K, V=V, N=B if cu is None else cu.numel() - 1,
        io_dtype=code(d["q"].dtype), state_dtype=code(d["state_dtype"]), q=d["q"], k=d["k"],
        v=d["v"], o=d["v"], cu_seqlens=cu, segment_tokens=segment_tokens))


def test_the_device_oracle_is_the_oracle():
    for lens in (None, [40, 0, 23]):
        d = inputs(1 if lens else 2, 63, 4, 2, 64, 128, "bf16", "fp32", "both", lens=lens)
        for a, b in zip(exact(d), oracle(d)):
            b = np.asarray(b)
            assert np.max(np.abs(a.cpu().numpy() - b)) <= 1e-12 * np.max(np.abs(b))


# more than 128 heads' worth of 64-row workgroups: two rounds of them, one of 128-row ones
@pytest.mark.parametrize("seg", [-1, 64, 320])
@pytest.mark.parametrize("B,T,H,Hk,K,V", [
    (1, 200, 130, 65, 64, 128), (1, 333, 130, 130, 128, 128), (3, 1000, 44, 4, 128, 128),
    (2, 449, 33, 11, 64, 256), (1, 1025, 44, 44, 128, 384),
])
def test_128_row_workgroups(B, T, H, Hk, K, V, seg):
    d = inputs(B, T, H, Hk, K, V, "bf16", "bf16", "g", seed=20)
    p = plan(d, seg)
    assert p["value_block"] == 128 and p["segment_tokens"] == (seg if 0 < seg < T else 0)
    o, s = run(d, segment_tokens=seg)
    check(o, s, exact(d), d, f"128 rows {B, T, H, Hk, K, V} seg {seg}")


LENS = [300, 1, 0, 129, 64, 515, 63]


@pytest.mark.parametrize("seg", [-1, 128, 256])
@pytest.mark.parametrize("K", [64, 128])
def test_128_row_workgroups_packed(K, seg):
    d = inputs(1, sum(LENS), 20, 5, K, 128, "bf16", "bf16", "io", lens=LENS, seed=21)
    assert plan(d, seg)["value_block"] == 128
    o, s = run(d, segment_tokens=seg)
    check(o, s, exact(d), d, f"128 rows packed K={K} seg {seg}")


@pytest.mark.parametrize("io,st", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"),
                                   ("fp32", "bf16")])
@pytest.mark.parametrize("T,seg", [(1600, 512), (1985, 192), (700, 576)])
@pytest.mark.parametrize("K,V", [(128, 64), (64, 128)])
def test_long_segments(T, seg, io, st, K, V):
    """Three to nine chunks in a segment: the rings of both launches wrap."""
    d = inputs(1, T, 3, 1, K, V, io, st, "both", seed=22)
    p = plan(d, seg)
    assert p["segment_tokens"] == seg and p["value_block"] == 64
    o, s = run(d, segment_tokens=seg)
    check(o, s, exact(d), d, f"long segments T={T} seg {seg} {io} {st} K={K}")


# calls that the automatic rule cuts into segments, and those past one round of workgroups
@pytest.mark.parametrize("B,T,H,K,V,io,st,lens,rows", [
    (1, 2048, 6, 128, 128, "bf16", "bf16", None, 64),
    (1, 4100, 3, 64, 64, "bf16", "fp32", None, 64),
    (2, 1999, 12, 128, 128, "fp32", "fp32", None, 64),      # one round of workgroups
    (1, 1999, 48, 128, 128, "fp32", "fp32", None, 64),      # two
    (1, 8192, 40, 128, 128, "bf16", "bf16", None, 128),     # past the last-level cache
    (1, 6001, 4, 128, 128, "bf16", "bf16", [4000, 0, 1, 2000], 64),
    (1, 3001, 3, 128, 128, "fp32", "fp32", [1500, 700, 801], 64),
])
def test_automatic_segments(B, T, H, K, V, io, st, lens, rows):
    d = inputs(B, T, H, H, K, V, io, st, "g", lens=lens, seed=23)
    p = plan(d)
    assert p["segment_tokens"] > 0 and p["value_block"] == rows, p
    o, s = run(d)
    check(o, s, exact(d), d, f"automatic B={B} T={T} H={H} {io} seg {p['segment_tokens']}")


@pytest.mark.parametrize("seg", [0, -1, 64, 192])
@pytest.mark.parametrize("K,V,st", [(128, 128, "fp32"), (64, 192, "bf16")])
def test_packed_fp32(K, V, st, seg):
    d = inputs(1, sum(LENS), 2, 1, K, V, "fp32", st, "g", lens=LENS, seed=24)
    o, s = run(d, segment_tokens=seg)
    check(o, s, exact(d), d, f"packed fp32 K={K} V={V} seg {seg}")


@pytest.mark.parametrize("io,st,H", [("bf16", "bf16", 2), ("bf16", "bf16", 20), ("bf16", "fp32", 3),
                                     ("fp32", "fp32", 2)])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("seg", [-1, 128])
def test_prompts_from_and_into_pool_slots(io, st, H, packed, seg):
    """Padded slots; one slot read by two sequences; an id outside read, one outside written;
    then the slots read are written. Everything else in the pool keeps its bits."""
    import torch

    T = sum(LENS) if packed else 290
    B, N = (1, len(LENS)) if packed else (7, 7)
    V = K = 128
    d = inputs(B, T, H, 1, K, V, io, st, "g", lens=LENS if packed else None, seed=25, state=False)
    assert plan(d, seg)["value_block"] == (128 if H == 20 else 64)
    base = torch.randn(16, H + 1, V, K, device="cuda").to(d["state_dtype"])
    pool = base[:, :H]
    frozen = base.clone()
    first = lambda ids: torch.stack([frozen[i, :H] if 0 <= i < 16 else torch.zeros_like(frozen[0, :H])
                                     for i in ids])
    ids = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    src, dst = [9, 9, 3, -1, 12, 16, 5], [0, 1, 3, 7, 14, 10, -3]
    o, s = run(d, state_in=pool, ssm_state_indices=ids(src), state_out_indices=ids(dst),
               segment_tokens=seg)
    assert s is pool
    ref = exact(d, first(src))
    held = [n for n, i in enumerate(dst) if 0 <= i < 16]
    pick = lambda x: x[held]
    check(o, pool[[dst[n] for n in held]], (ref[0], pick(ref[1]), ref[2], pick(ref[3])), d,
          f"pool {io} {st} H={H} packed {packed} seg {seg}")
    for i in range(16):
        assert torch.equal(base[i, H:], frozen[i, H:])
        assert i in dst or torch.equal(base[i], frozen[i]), i
    base.copy_(frozen)
    same = [8, 0, 15, 5, 1, 11, 2]
    o, _ = run(d, state_in=pool, ssm_state_indices=ids(same), segment_tokens=seg)
    check(o, pool[same], exact(d, first(same)), d, f"pool in place {io} {st} H={H} seg {seg}")


@pytest.mark.parametrize("B,T,H,io,st,lens", [
    (1, 8192, 6, "bf16", "bf16", None), (1, 4096, 96, "bf16", "bf16", None),
    (1, 18001, 24, "bf16", "fp32", [4001, 1500, 500, 3000, 2500, 2000, 4000, 500]),
    (2, 1999, 12, "fp32", "fp32", None), (3, 1000, 44, "bf16", "bf16", None),
])
def test_large_calls_repeat_themselves(B, T, H, io, st, lens):
    """Bit for bit: nothing depends on the order in which waves or workgroups run."""
    import torch

    d = inputs(B, T, H, H, 128, 128, io, st, "g", lens=lens, seed=26)
    o, s = run(d)
    for _ in range(8):
        o2, s2 = run(d)
        assert torch.equal(o, o2) and torch.equal(s, s2)
