"""The expert layer and the linear layer with epilogue give the same bits on
every call: nothing depends on timing, on what the caches hold, on the
workspace's old contents or on what runs before."""
import pytest
import torch

import fine_grained_fp8_token_b200 as fg
import workloads
from parity import F32, UE8M0, require_gpu
from test_gpu_moe_decode import route, weights_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    fg.load()
    return d


@pytest.mark.parametrize("fmt", [F32, UE8M0])
@pytest.mark.parametrize("T,E,topk,K,I", [(5, 8, 2, 1024, 384), (7, 16, 8, 2048, 512), (40, 12, 4, 1024, 384)])
def test_experts(dev, T, E, topk, K, I, fmt):
    W = weights_for(dev, E, K, I, fmt, seed=T)
    X = workloads.activations((T, K), "normal", seed=T).to(dev)
    ids, w = (t.to(dev) for t in route(T, E, topk, seed=1, holes=0.2))
    ws = torch.empty(fg.moe_workspace_bytes(T, topk, K, I), dtype=torch.uint8, device=dev)
    first = fg.moe_decode(X, ids, w, *W, fmt, residual=X)
    noise = torch.empty(200 << 20, dtype=torch.uint8, device=dev)
    for i in range(40):
        if i % 4 == 0:
            noise.fill_(i)                               # the caches' contents, and a long kernel before
        ws.fill_(255 - i)
        assert torch.equal(fg.moe_decode(X, ids, w, *W, fmt, residual=X, workspace=ws), first), i
    fg.check_device_status()


@pytest.mark.parametrize("M", [1, 30, 300])
def test_linear(dev, M):
    N, K, fmt = 512, 4096, F32
    X = workloads.activations((M, K), "normal", seed=M).to(dev)
    Wq, Ws = fg.quant_weight(workloads.weights((N, K), seed=1).to(dev), fmt)
    R = workloads.activations((M, N), "normal", seed=2).to(dev)
    first = fg.linear_epilogue(X, Wq, Ws, fmt, act="gelu", residual=R)
    noise = torch.empty(200 << 20, dtype=torch.uint8, device=dev)
    for i in range(40):
        if i % 4 == 0:
            noise.fill_(i)
        assert torch.equal(fg.linear_epilogue(X, Wq, Ws, fmt, act="gelu", residual=R), first), i
    fg.check_device_status()
