"""The router where the two largest keys of a group cancel (a bias that pins one
expert of a group and all but bans the others): the group's score is about 1
while its keys, and so the error of their 32-bit forms, are large.  Keys and
group scores are compared as in 64 bits, so the ids equal the definition's."""
import numpy as np
import pytest
import torch

import fine_grained_fp8_token_b200 as fg
from parity import require_gpu
from test_gpu_route import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    fg.load()
    return d


@pytest.mark.parametrize("B", [100.0, 1000.0, 10000.0, 1e6])
@pytest.mark.parametrize("G,keep,per", [(2, 1, 2), (8, 4, 4), (8, 3, 32)])
def test_keys_that_cancel(dev, B, G, keep, per):
    """Scores apart by a few steps of the 32-bit keys, and by less than one."""
    g = torch.Generator().manual_seed(int(B) + G + per)
    E, T = G * per, 300
    b = torch.full((E,), -4 * B)
    b[::per], b[1::per] = B, -B
    step = B * 2.0 ** -23
    z = torch.randn(T, 1, generator=g) + torch.randn(T, E, generator=g) * torch.tensor([step, 8 * step, 0.5])[:, None, None].repeat(
        1, T // 3, 1).reshape(T, 1)
    check(dev, z, min(4, E), score="sigmoid", bias=b, G=G, keep=keep)
    # the pinned and the banned expert at other places in every group, and several sizes of bias among the groups
    for i in range(G):
        b[i * per:(i + 1) * per] = b[i * per:(i + 1) * per][torch.randperm(per, generator=g)] * (1 + i % 3)
    check(dev, z, min(4, E), score="sigmoid", bias=b, G=G, keep=keep)


def test_infinite_and_overflowing_biases(dev):
    """+inf pins an expert for good; sums that leave fp32's range are decided in
    64 bits; a group whose every expert is off scores below all others."""
    g = torch.Generator().manual_seed(5)
    z = torch.randn(40, 32, generator=g)
    z[3, 8:16] = -np.inf
    z[4, :24] = -np.inf
    b = torch.randn(32, generator=g)
    for at, v in ((1, float("inf")), (9, 3e38), (10, 3e38), (17, 3e38), (18, -3e38), (25, -3e38)):
        b[at] = v
    for keep in (1, 2, 3):
        check(dev, z, 4, score="sigmoid", bias=b, G=4, keep=keep)
