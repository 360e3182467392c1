"""Sigmoid weights at the far end: sigma(z) below fp32's normal numbers
(z < -87.3) and past the exponential's overflow (z < -88.7).  They keep what
fp32 holds of them: exp is off by at most one step there, 2^-149, which the
division by the least sum, 1e-20, turns into 2^-149 / 1e-20."""
import numpy as np
import pytest
import torch

import fine_grained_fp8_token_b200 as fg
from parity import require_gpu
from test_gpu_route import check, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    fg.load()
    return d


@pytest.mark.parametrize("lo,hi", [(-30, -20), (-88, -80), (-95, -86), (-103, -93), (-120, -100)])
@pytest.mark.parametrize("biased", [False, True])
def test_vanishing_sigmoids(dev, lo, hi, biased):
    g = torch.Generator().manual_seed(-lo)
    z = torch.rand(64, 48, generator=g) * (hi - lo) + lo
    b = torch.rand(48, generator=g) if biased else None
    check(dev, z, 6, score="sigmoid", bias=b, renorm=False)
    ids, w = fg.route_topk(z.to(dev), 6, score="sigmoid", bias=None if b is None else b.to(dev))
    ri, rw = reference(z, 6, "sigmoid", b, 1, 1, True, 1.0)
    assert (ids.cpu().numpy() == ri).all()
    assert (np.abs(w.double().cpu().numpy() - rw) <= 2.0 ** -19 * rw + 2.0 ** -149 / 1e-20).all()
