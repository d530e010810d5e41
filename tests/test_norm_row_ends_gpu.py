"""Norms of rows that end inside a thread's chunk of channels: every remainder, with NaN between the rows, which no result
may have."""
import pytest
import torch

from test_norms_gpu import BF, IDS, TYPES, check, tensors

pytestmark = pytest.mark.gpu


def apart(t, pad):
    """The same rows, `pad` NaN elements before each."""
    if t is None or t.dim() != 2:
        return t
    room = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), device="cuda", dtype=t.dtype)
    room[:, pad:] = t
    return room[:, pad:]


@pytest.mark.parametrize("tx,ty", TYPES, ids=IDS)
@pytest.mark.parametrize("gate", ["vector", "matrix"])
@pytest.mark.parametrize("d", [*range(1, 10), 121, *range(129, 137), 507, *range(513, 518), 767, 773, 1026, 1531, 1539, 2047,
                               4093, 4100, 8187, 8193, 16377])
def test_every_remainder(d, gate, tx, ty):
    x, y, kw = tensors(5, d, tx, ty, seed=d, gate=gate)
    kw["gate"] = apart(kw["gate"], 3)
    check(apart(x, 5), apart(y, 3), **kw)


@pytest.mark.parametrize("d", [131, 516, 1027])
def test_scale_of_channels(d):
    x, y, kw = tensors(700, d, BF, BF, seed=d, scale="vector", gate=None)
    check(apart(x, 1), apart(y, 2), **kw)
