"""kda_short_conv with offsets past 32 bits: sequences and slots more than 2^31 elements apart,
and a call of more than 2^31 elements. Tolerances as in test_gpu_short_conv.py."""

import numpy as np
import pytest

from test_gpu_short_conv import _gpu, check_out, host, inputs, oracle, run  # noqa: F401

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
