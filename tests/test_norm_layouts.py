"""The row strides that the gated norm's binding hands to the C entry point: every row that
they name lies in the tensor and is that row. PyTorch calls a tensor contiguous whatever the
strides of its axes of one entry are, so those strides must not be used. CPU only."""

import math

import pytest

torch = pytest.importorskip("torch")

from chunkwise_delta_rule_kda_amd import _tensors  # noqa: E402
from chunkwise_delta_rule_kda_amd.norm import _rows  # noqa: E402

_tensors.get_torch()


def tensor(*shape):
    return torch.arange(math.prod(shape), dtype=torch.float32).view(*shape)


LAYOUTS = {
    "one token of a sequence-first model": lambda: tensor(1, 5, 4, 128).transpose(0, 1),
    "one token, heads and tokens exchanged": lambda: tensor(2, 3, 1, 128).transpose(1, 2),
    "one head": lambda: tensor(1, 6, 1, 64).transpose(0, 1).transpose(1, 2),
    "one token of one head": lambda: tensor(1, 7, 64)[:, :, None].permute(1, 0, 2, 3),
    "three axes, the first of one entry": lambda: tensor(4, 1, 64).transpose(0, 1),
    "three axes, the second of one entry": lambda: tensor(1, 4, 64).transpose(0, 1),
    "five axes with two of one entry": lambda: tensor(1, 1, 3, 2, 64).permute(2, 0, 1, 3, 4),
    "a size-1 axis with any stride": lambda: torch.as_strided(tensor(768), (2, 1, 3, 128),
                                                              (384, 5, 128, 1)),
    "dense": lambda: tensor(2, 3, 4, 64),
    "two axes": lambda: tensor(5, 64),
    "one row": lambda: tensor(64),
    "slice of a projection": lambda: tensor(2, 3, 5, 4, 72)[:, :, 2, :, :64],
    "one token of a slice": lambda: tensor(5, 3, 5, 4, 72)[:, :1, 2, :, :64],
    "one gate for all heads": lambda: tensor(2, 3, 1, 64).expand(2, 3, 4, 64),
    "no rows": lambda: tensor(0, 4, 64),
}


@pytest.mark.parametrize("name", LAYOUTS)
def test_rows_are_the_tensors_own(name):
    t = LAYOUTS[name]()
    D = t.shape[-1]
    G = t.shape[-2] if t.dim() > 2 else 1
    M = t.numel() // (D * G)
    m, g = _rows(t, "t")
    flat = t.reshape(M, G, D)
    last = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
    for i in range(M):
        for j in range(G):
            at = i * m + j * g
            assert at + D <= last, (name, i, j, m, g)
            row = torch.as_strided(t, (D,), (1,), t.storage_offset() + at)
            assert torch.equal(row, flat[i, j]), (name, i, j, m, g)
    assert m % 8 == 0 and g % 8 == 0  # what the C entry point asks of them
