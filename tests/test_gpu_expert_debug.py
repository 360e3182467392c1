"""The epilogue GEMM, the router and the few-token expert layer in the
index-checking build: no check fails, and the bits are those of the release
build."""
import ctypes

import pytest
import torch

import fine_grained_fp8_token_b200 as fg
import workloads
from fine_grained_fp8_token_b200 import build as fgbuild
from parity import F32, UE8M0, Guarded, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    require_gpu()
    release = fg.load()
    debug = ctypes.CDLL(fgbuild.build(debug=True))
    for name, (res, args) in fg.SIGNATURES.items():
        fn = getattr(debug, name)
        fn.restype, fn.argtypes = res, args
    return release, debug


def both(libs, monkeypatch, fn):
    outs = []
    for lib in libs:
        with monkeypatch.context() as mp:
            mp.setattr(fg, "load", lambda build_if_missing=True: lib)
            outs.append(fn())
            fg.check_device_status()
    for x, y in zip(*outs):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("fmt", [F32, UE8M0])
@pytest.mark.parametrize("M,N,K", [(1, 1280, 1024), (7, 128, 384), (16, 4096, 256), (64, 640, 7168), (65, 384, 512),
                                   (300, 640, 2048), (1200, 4096, 256)])
def test_linear_epilogue(libs, monkeypatch, M, N, K, fmt):
    dev = torch.device("cuda:0")
    X = workloads.activations((M, K), "normal_outliers", seed=M, device=dev)
    W = workloads.weights((N, K), seed=N, device=dev)
    b = torch.linspace(-1, 1, N, device=dev)
    R = workloads.activations((M, N), "normal", seed=K, device=dev)

    def run():
        Wq, Ws = fg.quant_weight(W, fmt)
        Xq, Xs = fg.quant_act(X, fmt)
        out = [Guarded((M, N), torch.bfloat16, dev) for _ in range(2)]
        fg.linear_epilogue(X, Wq.view(torch.float8_e4m3fn), Ws, fmt, bias=b, act="gelu", residual=R, Y=out[0].t)
        fg.gemm_epilogue(Xq, Xs, Wq, Ws, fmt, bias=b.bfloat16(), act="silu", Y=out[1].t)
        torch.cuda.synchronize()
        for o in out:
            o.check()
        return [o.t for o in out]
    both(libs, monkeypatch, run)


@pytest.mark.parametrize("fmt", [F32, UE8M0])
@pytest.mark.parametrize("T,E,topk,K,I", [(1, 8, 8, 640, 256), (16, 40, 4, 256, 384), (17, 5, 2, 384, 128),
                                          (64, 12, 6, 512, 256)])
def test_routing_and_experts(libs, monkeypatch, T, E, topk, K, I, fmt):
    dev = torch.device("cuda:0")
    X = workloads.activations((T, K), "normal", seed=T, device=dev)
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(E)).to(dev)
    z[T // 2, E // 2:] = -float("inf")
    W = [workloads.weights(s, seed=i, device=dev) for i, s in enumerate([(E * 2 * I, K), (E * K, I)])]

    def run():
        W13q, W13s = fg.quant_weight(W[0], fmt)
        W2q, W2s = fg.quant_weight(W[1], fmt)
        ids, w = fg.route_topk(z, topk, score="sigmoid", bias=torch.linspace(0, 1, E, device=dev))
        Y = Guarded((T, K), torch.bfloat16, dev)
        ws = Guarded((fg.moe_workspace_bytes(T, topk, K, I),), torch.uint8, dev)
        fg.moe_decode(X, ids, w, W13q.view(E, 2 * I, K), W13s.view(E, 2 * I // 128, K // 128), W2q.view(E, K, I),
                      W2s.view(E, K // 128, I // 128), fmt, residual=X, Y=Y.t, workspace=ws.t)
        torch.cuda.synchronize()
        Y.check()
        ws.check("workspace")
        return [ids, w, Y.t]
    both(libs, monkeypatch, run)
