"""The few-token kernels' own unwinding on the GPU, without a fault: one weight
tile of CTA 0 is never requested, so its roles' bounded waits expire, then those
of the ranks that meet with it, and the launch ends within seconds with
FGFP8_ERR_TIMEOUT.  The other clusters' output is correct, and the next call on
the same context is correct everywhere."""
import time

import pytest
import torch

import fine_grained_fp8_token_b200 as fg
import oracle
import workloads
from parity import F32, UE8M0, assert_gemm_close, require_gpu, to_np, y_to_f64

pytestmark = pytest.mark.gpu
TIMEOUT = 6


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    fg.load()
    return d


def expired(call):
    """Runs the call, which must end with a timeout within a minute."""
    fg.check_device_status()
    t0 = time.monotonic()
    assert call() == 0
    with pytest.raises(fg.FGFP8Error) as ei:
        fg.check_device_status()
    waited = time.monotonic() - t0
    assert ei.value.status == TIMEOUT
    assert 0.9 < waited < 60.0, waited
    fg.check_device_status()                            # the read cleared the word


# one token tile of 16 and one of 64, K blocks of a rank below and above the
# stages (N = 512: four clusters of eight ranks)
@pytest.mark.parametrize("M,K,withhold,fmt", [(5, 4096, 1, F32), (40, 4096, 0, UE8M0), (5, 16384, 6, UE8M0), (40, 20480, 9, F32)])
def test_linear(dev, M, K, withhold, fmt):
    N = 512
    cfg = workloads.scaled_linear(workloads.TINY, M=M, N=N, K=K, seed=M + K)
    X, W = workloads.linear_inputs(cfg)
    Xq, Xs = fg.quant_act(X.to(dev), fmt)
    Wq, Ws = fg.quant_weight(W.to(dev), fmt)
    Y = torch.zeros(M, N, dtype=torch.bfloat16, device=dev)
    expired(lambda: fg.fgfp8_selftest_few_timeout(Xq.data_ptr(), Xs.data_ptr(), Xs.shape[1], Wq.data_ptr(), Ws.data_ptr(),
                                                  Y.data_ptr(), M, N, K, fmt, withhold,
                                                  torch.cuda.current_stream().cuda_stream))
    ref, S = oracle.gemm(to_np(Xq), to_np(Xs), to_np(Wq), to_np(Ws), fmt)
    assert_gemm_close(y_to_f64(Y)[:, 128:], ref[:, 128:], S[:, 128:], "the other clusters' columns")
    again = fg.gemm_epilogue(Xq, Xs, Wq, Ws, fmt)
    fg.check_device_status()
    assert_gemm_close(y_to_f64(again), ref, S, "after the unwound launch")


# gate/up with shared items alone, and with items of its CTAs' own before them
# (more than one round); down in ranks that meet eight tokens at a time, and all at once
@pytest.mark.parametrize("T,E,topk,K,I,kernel,withhold", [(6, 4, 2, 1024, 512, 0, 1), (6, 4, 2, 1024, 512, 1, 1),
                                                         (40, 4, 2, 1024, 512, 0, 0), (40, 4, 2, 1024, 512, 1, 0),
                                                         (8, 16, 8, 256, 2560, 0, 1), (40, 16, 4, 512, 1536, 0, 2)])
def test_experts(dev, T, E, topk, K, I, kernel, withhold):
    fmt = F32
    X = workloads.activations((T, K), "normal", seed=T).to(dev)
    W13q, W13s = fg.quant_weight(workloads.weights((E * 2 * I, K), seed=1, device=dev), fmt)
    W2q, W2s = fg.quant_weight(workloads.weights((E * K, I), seed=2, device=dev), fmt)
    ids = torch.stack([torch.arange(topk, dtype=torch.int32) * (E // topk) + t % (E // topk) for t in range(T)]).to(dev)
    w = torch.full((T, topk), 1.0 / topk, device=dev)
    W = (W13q.view(E, 2 * I, K), W13s.view(E, 2 * I // 128, K // 128), W2q.view(E, K, I), W2s.view(E, K // 128, I // 128))
    good = fg.moe_decode(X, ids, w, *W, fmt)
    Y = torch.zeros_like(good)
    ws = torch.empty(fg.moe_workspace_bytes(T, topk, K, I), dtype=torch.uint8, device=dev)
    expired(lambda: fg.fgfp8_selftest_moe_timeout(
        X.data_ptr(), K, ids.data_ptr(), w.data_ptr(), *(t.data_ptr() for t in W), Y.data_ptr(), ws.data_ptr(), ws.numel(),
        T, topk, E, K, I, fmt, kernel, withhold, torch.cuda.current_stream().cuda_stream))
    if kernel == 1:
        assert torch.equal(Y[:, 128:], good[:, 128:])       # columns of the other clusters
    assert torch.equal(fg.moe_decode(X, ids, w, *W, fmt, workspace=ws), good)
    fg.check_device_status()


@pytest.mark.parametrize("M", [5, 40])
def test_a_tile_beyond_the_share_withholds_nothing(dev, M):
    N, K, fmt = 512, 4096, F32
    cfg = workloads.scaled_linear(workloads.TINY, M=M, N=N, K=K, seed=3)
    X, W = workloads.linear_inputs(cfg)
    Xq, Xs = fg.quant_act(X.to(dev), fmt)
    Wq, Ws = fg.quant_weight(W.to(dev), fmt)
    Y = torch.zeros(M, N, dtype=torch.bfloat16, device=dev)
    assert fg.fgfp8_selftest_few_timeout(Xq.data_ptr(), Xs.data_ptr(), Xs.shape[1], Wq.data_ptr(), Ws.data_ptr(),
                                         Y.data_ptr(), M, N, K, fmt, 31, torch.cuda.current_stream().cuda_stream) == 0
    fg.check_device_status()
    assert torch.equal(Y, fg.gemm_epilogue(Xq, Xs, Wq, Ws, fmt))
