"""Slots of a state pool: copies, forks, restores, clears and compaction. Results are exact:
a slot's bits are moved, an FP32 value that goes into a BF16 pool is rounded to nearest
even (torch's own conversion), a BF16 value widens exactly."""

import numpy as np
import pytest

from oracle import compact_slots

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import chunkwise_delta_rule_kda_amd as kda

    kda.load_library()


def ids(x):
    import torch

    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def dtype(n):
    import torch

    return {"bf16": torch.bfloat16, "fp32": torch.float32}[n]


def expected(pool, source, src, dst):
    """Pair by pair, from the contents before the call."""
    import torch

    out, source = pool.clone(), source.clone()
    for a, b in zip(src, dst):
        if 0 <= b < pool.shape[0]:
            held = 0 <= a < source.shape[0]
            out[b] = source[a].to(pool.dtype) if held else torch.zeros_like(out[b])
    return out


# sizes around a workgroup's 8192 elements, and the smallest
@pytest.mark.parametrize("shape", [(8,), (1, 128, 128), (3, 64, 128), (8192,), (8200,), (8184,),
                                   (2, 8192)])
@pytest.mark.parametrize("sd,dd", [("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "bf16"),
                                   ("bf16", "fp32")])
def test_copy(shape, sd, dd):
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    torch.manual_seed(0)
    pool = torch.randn(11, *shape, device="cuda").to(dtype(dd))
    source = torch.randn(6, *shape, device="cuda").to(dtype(sd))
    src = [0, 5, 5, 5, -1, 3, 6, 2**31 - 1, 2]   # a fork of 5, three sources outside
    dst = [4, 0, 1, 10, 2, -1, 3, 9, 11]         # two destinations outside
    want = expected(pool, source, src, dst)
    got = kda.kda_pool_copy(pool, ids(src), ids(dst), source=source)
    torch.cuda.synchronize()
    assert got is pool and torch.equal(pool, want)


def test_special_values_are_moved_and_rounded():
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    x = torch.tensor([0.0, -0.0, 1.00390625, 1.01171875, 3.4e38, -3.4e38, float("inf"),
                      float("-inf"), 1e-40, float("nan"), 65504.0, 1.0, -1.0, 2.0, 5.9e-39, 7.0],
                     device="cuda")
    src = x.view(1, 16)
    for d in ("bf16", "fp32"):
        pool = torch.ones(2, 16, device="cuda").to(dtype(d))
        kda.kda_pool_copy(pool, ids([0]), ids([1]), source=src)
        a, b = pool[1], x.to(dtype(d))
        assert torch.equal(a.nan_to_num(5), b.nan_to_num(5)) and torch.equal(a.isnan(), b.isnan())
        assert torch.equal(torch.signbit(a)[:9], torch.signbit(b)[:9])


def test_within_one_pool():
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    pool = torch.randn(9, 2, 128, 128, device="cuda")
    src, dst = [1, 1, 4, 6, -5], [0, 2, 3, 6, 8]   # 6 onto itself
    want = expected(pool, pool, src, dst)
    kda.kda_pool_copy(pool, ids(src), ids(dst))
    assert torch.equal(pool, want)
    kda.kda_pool_copy(pool, ids([]), ids([]))
    assert torch.equal(pool, want)


@pytest.mark.parametrize("sd,dd", [("bf16", "bf16"), ("fp32", "bf16")])
def test_layers_and_padding(sd, dd):
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    L, H = 3, 2
    base = torch.randn(L, 8, H + 1, 128, 64, device="cuda").to(dtype(dd))
    frozen = base.clone()
    pool = base[:, 1:7, :H]                       # padded slots and layers
    source = torch.randn(5, L, H, 128, 64, device="cuda").to(dtype(sd)).transpose(0, 1)
    src, dst = [4, 4, 0, 9], [0, 5, 2, 3]         # source: layers inside the slots' pitch
    want = frozen.clone()
    for l in range(L):
        want[l, 1:7, :H] = expected(frozen[l, 1:7, :H], source[l], src, dst)
    kda.kda_pool_copy(pool, ids(src), ids(dst), source=source, layered=True)
    torch.cuda.synchronize()
    assert torch.equal(base, want)


def test_long_pool_offsets():
    """Slots past 2^31 elements from the base."""
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    pool = torch.empty(1100, 2 ** 21, dtype=torch.bfloat16, device="cuda")
    for i in (0, 1, 1099):
        pool[i] = i + 1
    kda.kda_pool_copy(pool, ids([1099, 0]), ids([5, 1098]))
    assert bool((pool[5] == 1100).all()) and bool((pool[1098] == 1).all())
    new, count = kda.kda_pool_compact(pool, ids([1099, 1]))
    assert new.tolist() == [0, 1] and count.item() == 2
    assert bool((pool[0] == 1100).all()) and bool((pool[1] == 2).all())


def test_checkpoints_restored_into_a_pool():
    """Rows of kda_prefill's checkpoint buffer as the source."""
    import torch

    import chunkwise_delta_rule_kda_amd as kda
    import kda_synth
    from kda_testlib import to_device

    x = kda_synth.config(2, T=96, H=2)
    d = to_device(x)
    q, k, v, g, beta = (d.pop(n) for n in ("q", "k", "v", "g", "beta"))
    _, _, ck = kda.kda_prefill(q, k, v, g, beta, checkpoint_every=32, **d)
    pool = torch.zeros(4, 2, 128, 128, device="cuda")
    kda.kda_pool_copy(pool, ids([2, 1]), ids([3, 0]), source=ck)
    assert torch.equal(pool[3], ck[2].float()) and torch.equal(pool[0], ck[1].float())
    assert not pool[1].any() and not pool[2].any()


def compact_case(pool, slots, in_place=False, **kw):
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    n = pool.shape[0]
    before = pool.clone()
    new, count, moves = compact_slots(slots, n)
    t = ids(slots)
    got, c = kda.kda_pool_compact(pool, t, new_slots=t if in_place else None, **kw)
    torch.cuda.synchronize()
    assert got.tolist() == new and c.item() == count
    want = before.clone()
    for a, b in moves.items():
        want[b] = before[a]
    assert torch.equal(pool, want)
    for i, j in zip(slots, new):  # every live slot keeps its contents
        if 0 <= i < n:
            assert torch.equal(pool[j], before[i])


@pytest.mark.parametrize("slots", [[], [0], [7], [7, 6, 5, 4], [0, 1, 2], [3, 3, 3, 7], [0, 7, 2, 5],
                                   [-1, 6, 8, 99, 1], list(range(8)), [2**31 - 1, -2**31, 5]])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(slots, in_place):
    import torch

    torch.manual_seed(1)
    compact_case(torch.randn(8, 2, 64, 64, device="cuda"), slots, in_place)


@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 1000, 40000, 1 << 18])
def test_compact_random(n):
    import torch

    rng = np.random.default_rng(n)
    pool = torch.arange(n * 8, device="cuda", dtype=torch.float32).view(n, 8)
    for share in (0.03, 0.5, 0.97):
        k = max(1, int(n * share))
        slots = rng.permutation(n)[:k].tolist()
        compact_case(pool.clone(), slots + slots[:3])


def test_compact_layers():
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    pool = torch.randn(3, 10, 1, 128, 128, device="cuda").bfloat16()
    before = pool.clone()
    new, count = kda.kda_pool_compact(pool, ids([9, 1, 8]), layered=True)
    assert new.tolist() == [2, 1, 0] and count.item() == 3
    assert torch.equal(pool[:, 0], before[:, 8]) and torch.equal(pool[:, 2], before[:, 9])
    assert torch.equal(pool[:, 3:], before[:, 3:])


def test_graphs():
    """A captured fork and a captured compaction, replayed with new ids in place and eager
    work in between."""
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    torch.manual_seed(2)
    first = torch.randn(12, 2, 128, 128, device="cuda")
    pool, src, dst = first.clone(), ids([0, 0, 0]), ids([1, 2, 3])
    live, new, count = ids([9, 4, 2]), ids([0, 0, 0]), ids([0])
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        kda.kda_pool_copy(pool, src, dst)
        kda.kda_pool_compact(pool, live, new_slots=new, count=count, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_pool_copy(pool, src, dst)
        kda.kda_pool_compact(pool, live, new_slots=new, count=count, workspace=ws)
    for a, b, slots in (([0, 0, 0], [1, 2, 3], [9, 4, 2]), ([5, -1, 5], [7, 8, 11], [11, 7, 3]),
                        ([3, 3, 3], [6, 6, 6], [0, 1, 2])):
        b = b if len(set(b)) == 3 else [6, -1, -1]
        src.copy_(ids(a)), dst.copy_(ids(b)), live.copy_(ids(slots))
        pool.copy_(first)
        other = torch.randn(12, 2, 64, 64, device="cuda")
        compact_case(other, slots)  # eager, with a workspace of its own
        want = expected(first, first, a, b)
        to, n, moves = compact_slots(slots, 12)
        held = want.clone()
        for i, j in moves.items():
            want[j] = held[i]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool, want) and new.tolist() == to and count.item() == n


def test_other_stream():
    import torch

    import chunkwise_delta_rule_kda_amd as kda

    pool = torch.randn(8, 2, 128, 128, device="cuda")
    want = expected(pool, pool, [1], [7])
    a, b, live = ids([1]), ids([7]), ids([7, 6])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kda.kda_pool_copy(pool, a, b, stream=side)
    side.synchronize()
    assert torch.equal(pool, want)
    new, count = kda.kda_pool_compact(pool, live, stream=side.cuda_stream)
    side.synchronize()
    assert new.tolist() == [1, 0] and count.item() == 2
    assert torch.equal(pool[1], want[7]) and torch.equal(pool[0], want[6])
