"""The activations' tails in the GEMM's epilogue, relative to the value: x comes
through the bias (X = 0), so the output is bf16(act(x)).

Tolerance, before the run: half a bf16 step, 2^-8 |y|, and the activation's own
error.  silu and gelu_tanh: exp(-z) from its fp32 argument is off by a few
|z| 2^-24, 2^-15 for |z| <= 88; where 1 + exp(-z) passes 2^126 its reciprocal
is flushed, |y| < 2^7 2^-126.  gelu: 2^-16 (the fit 2^-20, the argument a^2 / 2
<= 87 of its exponential two roundings, the rest a few 2^-23); below fp32's
normal numbers flushed."""
import math

import pytest
import torch

import fine_grained_fp8_token_b200 as fg
import workloads
from parity import F32, UE8M0, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    fg.load()
    return d


def act64(x, act):
    if act == "relu":
        return x.clamp(min=0)
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return x * 0.5 * torch.special.erfc(-x / math.sqrt(2))
    if act == "gelu_tanh":
        return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    return x


OWN = {"none": (0.0, 0.0), "relu": (0.0, 0.0), "silu": (2.0 ** -15, 2.0 ** -119), "gelu": (2.0 ** -16, 2.0 ** -126),
       "gelu_tanh": (2.0 ** -15, 2.0 ** -119)}


@pytest.mark.parametrize("fmt", [F32, UE8M0])
@pytest.mark.parametrize("M", [2, 40, 80])
@pytest.mark.parametrize("act", list(OWN))
def test_tails_relative_to_the_value(dev, act, M, fmt):
    N, K = 2048, 128
    x = torch.cat([torch.linspace(-15, 0, 1024), torch.linspace(0, 15, 256), torch.linspace(-130, -15, 256),
                   -torch.logspace(-36, 0, 256), torch.logspace(-36, 4, 256)])
    Wq, Ws = fg.quant_weight(workloads.weights((N, K), seed=1).to(dev), fmt)
    X = torch.zeros(M, K, dtype=torch.bfloat16, device=dev)
    y = fg.linear_epilogue(X, Wq, Ws, fmt, bias=x.to(dev), act=act).double().cpu()
    fg.check_device_status()
    ref = act64(x.double(), act)
    rel, floor = OWN[act]
    off = (y - ref).abs() - ((2.0 ** -8 + rel) * ref.abs() + floor + 2.0 ** -134)
    bad = (off > 0).any(dim=0)
    assert not bad.any(), f"{int(bad.sum())} of {N}, first at x = {x[bad][0].item()}: {y[0, bad][0].item()} for {ref[bad][0].item()}"
    assert (y[:, x < 0] <= 0).all()
    assert (y == y[:1]).all()
