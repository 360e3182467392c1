"""GPU checks of the linear layer with its epilogue (fgfp8_gemm_epilogue,
fgfp8_linear_epilogue) against the formula in 64 bits on the oracle's codes.

Tolerance per element, before the run: the GEMM's own bound 1e-4 S on the sum
(S = sum_k |x_hat w_hat|) times the steepest slope of the activations (gelu:
1.13), the fp32 epilogue (a few steps of 2^-24 on sums of |acc| + |bias| +
|residual|, 2^-18 allowed) and the rounding of the result (half a bf16 step,
2^-8 |y|)."""
import math

import numpy as np
import pytest
import torch

import fine_grained_fp8_token_b200 as fg
import oracle
import workloads
from parity import Guarded, bits16, require_gpu, to_np, y_to_f64

pytestmark = pytest.mark.gpu
F32, UE8M0 = 0, 1
ERF = np.vectorize(math.erf)


@pytest.fixture(scope="module")
def dev():
    d = require_gpu()
    fg.load()
    return d


def act64(y, act):
    with np.errstate(over="ignore"):
        if act == "relu":
            return np.maximum(y, 0.0)
        if act == "silu":
            return y / (1 + np.exp(-y))
        if act == "gelu":
            return 0.5 * y * (1 + ERF(y / math.sqrt(2)))
        if act == "gelu_tanh":
            return 0.5 * y * (1 + np.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y


def make(dev, M, N, K, fmt, bias, residual, seed=0):
    X = workloads.activations((M, K), "normal_outliers", seed=seed)
    W = workloads.weights((N, K), seed=seed + 1)
    Wq, Ws = fg.quant_weight(W.to(dev), fmt)
    g = torch.Generator().manual_seed(seed + 2)
    b = None if bias is None else torch.randn(N, generator=g).to(bias)
    R = torch.randn(M, N, generator=g).to(torch.bfloat16) if residual else None
    return X, Wq, Ws, b, R


def reference(X, Wq, Ws, fmt, b, act, R, rows=None):
    Xq, Xs = oracle.quant_act(bits16(X), fmt)
    acc, S = oracle.gemm(Xq, Xs, to_np(Wq), to_np(Ws), fmt, rows=rows)
    bias = 0.0 if b is None else b.double().cpu().numpy()[None, :]
    r = 0.0 if R is None else (R if rows is None else R[rows]).double().cpu().numpy()
    y = act64(acc + bias, act) + r
    tol = 1.13e-4 * S + 2.0 ** -18 * (np.abs(acc) + np.abs(bias) + np.abs(r)) + 2.0 ** -8 * np.abs(y)
    return y, tol


def check(Y, ref, tol, what=""):
    got = y_to_f64(Y)
    bad = np.abs(got - ref) > tol
    assert np.isfinite(got).all() and not bad.any(), (
        f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[:1]}: {got[bad][:3]} {ref[bad][:3]}")


SHAPES = [(1, 128, 128), (1, 4096, 1024), (2, 256, 640), (3, 1152, 128), (15, 384, 512), (16, 512, 2048),
          (17, 128, 384), (33, 1280, 1024), (64, 640, 256), (65, 256, 512), (100, 384, 1024), (300, 768, 1280)]


@pytest.mark.parametrize("fmt", [F32, UE8M0])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_bias_activation_residual(dev, M, N, K, fmt):
    acts = ["none", "relu", "silu", "gelu", "gelu_tanh"]
    for n, act in enumerate(acts if M < 64 else acts[M % 5:M % 5 + 1] + ["none"]):
        bias = (None, torch.bfloat16, torch.float32)[(n + M) % 3]
        residual = (n + M + fmt) % 2 == 0
        X, Wq, Ws, b, R = make(dev, M, N, K, fmt, bias, residual, seed=M + n)
        out = Guarded((M, N), torch.bfloat16, dev)
        Y = fg.linear_epilogue(X.to(dev), Wq, Ws, fmt, bias=None if b is None else b.to(dev), act=act,
                               residual=None if R is None else R.to(dev), Y=out.t)
        fg.check_device_status()
        check(Y, *reference(X, Wq, Ws, fmt, b, act, R), f"linear {act} {bias} {residual}")
        out.check()
        Xq, Xs = fg.quant_act(X.to(dev), fmt)
        Y2 = fg.gemm_epilogue(Xq, Xs, Wq, Ws, fmt, bias=None if b is None else b.to(dev), act=act,
                              residual=None if R is None else R.to(dev))
        fg.check_device_status()
        check(Y2, *reference(X, Wq, Ws, fmt, b, act, R), f"gemm {act}")


@pytest.mark.parametrize("M", [1, 40, 200])
def test_strided_rows_and_residual_in_place(dev, M):
    """X and the residual as column slices of wider buffers; the residual
    being the output itself."""
    N, K, fmt = 512, 768, F32
    X, Wq, Ws, b, R = make(dev, M, N, K, fmt, torch.float32, True, seed=5)
    wide = torch.full((M, K + 136), 7.0, dtype=torch.bfloat16, device=dev)
    wide[:, 8:8 + K] = X.to(dev)
    rwide = torch.full((M, N + 64), 9.0, dtype=torch.bfloat16, device=dev)
    rwide[:, 16:16 + N] = R.to(dev)
    ref = reference(X, Wq, Ws, fmt, b, "silu", R)
    check(fg.linear_epilogue(wide[:, 8:8 + K], Wq, Ws, fmt, bias=b.to(dev), act="silu", residual=rwide[:, 16:16 + N]),
          *ref)
    Y = R.to(dev).clone()
    assert fg.linear_epilogue(X.to(dev), Wq, Ws, fmt, bias=b.to(dev), act="silu", residual=Y, Y=Y) is Y
    check(Y, *ref)
    fg.check_device_status()


def test_no_epilogue_equals_the_plain_layer(dev):
    """Without bias, activation and residual the prefill kernels give the plain
    GEMM's output bit for bit (the same sums, rounded once)."""
    for fmt in (F32, UE8M0):
        X, Wq, Ws, _, _ = make(dev, 300, 512, 1024, fmt, None, False, seed=9)
        a, b = fg.linear(X.to(dev), Wq, Ws, fmt), fg.linear_epilogue(X.to(dev), Wq, Ws, fmt)
        assert torch.equal(a, b)


def test_activation_tails(dev):
    """Far arguments of every activation, through the bias (x = 0): no NaN, no
    sign error, the tails' values."""
    N, K = 128, 128
    v = torch.tensor([0.0, -0.0, 1e-3, -1e-3, 0.5, -0.5, 3.0, -3.0, 5.5, -5.5, 9.0, -9.0, 50.0, -50.0, 90.0, -90.0, 1e4, -1e4,
                      1e30, -1e30])
    b = torch.zeros(N)
    b[:len(v)] = v
    Wq, Ws = fg.quant_weight(workloads.weights((N, K), seed=1).to(dev), F32)
    for M in (2, 80):
        X = torch.zeros(M, K, dtype=torch.bfloat16)
        for act in ("none", "relu", "silu", "gelu", "gelu_tanh"):
            got = y_to_f64(fg.linear_epilogue(X.to(dev), Wq, Ws, F32, bias=b.to(dev), act=act))
            ref = act64(b.double().numpy(), act)
            # half a bf16 step, and the erf formula's 1.5e-7 |x| / 2 in gelu's tail
            tol = 2.0 ** -8 * np.abs(ref) * 1.01 + 1.5e-7 * np.minimum(np.abs(b.double().numpy()), 10) + 1e-30
            assert (np.abs(got - ref[None]) <= tol).all(), (act, M, got[0], ref)
        nan = torch.full((N,), float("nan"))
        for act in ("none", "relu", "silu", "gelu", "gelu_tanh"):
            assert fg.linear_epilogue(X.to(dev), Wq, Ws, F32, bias=nan.to(dev), act=act).isnan().all()


def test_large_layer_sampled_rows(dev):
    """A wide prefill: the first and last row of M tiles against the oracle."""
    M, N, K = 1000, 4096, 4096
    X, Wq, Ws, b, R = make(dev, M, N, K, F32, torch.bfloat16, True, seed=3)
    Y = fg.linear_epilogue(X.to(dev), Wq, Ws, F32, bias=b.to(dev), act="gelu", residual=R.to(dev))
    fg.check_device_status()
    rows = np.array([0, 127, 128, 500, 895, 896, 999])
    ref, tol = reference(X, Wq, Ws, F32, b, "gelu", R, rows=rows)
    check(Y[torch.as_tensor(rows, device=dev)], ref, tol)


def test_side_stream_and_graph_replay(dev):
    """On a stream that is not current, and captured: a replay on new inputs
    gives the eager result."""
    for M in (4, 40, 200):
        X, Wq, Ws, b, R = make(dev, M, 384, 512, F32, torch.bfloat16, True, seed=M)
        Xd, Rd, bd = X.to(dev), R.to(dev), b.to(dev)
        eager = fg.linear_epilogue(Xd, Wq, Ws, F32, bias=bd, act="gelu", residual=Rd)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = fg.linear_epilogue(Xd, Wq, Ws, F32, bias=bd, act="gelu", residual=Rd, stream=side)
        side.synchronize()
        assert torch.equal(eager, other)
        buf, out = torch.zeros_like(Xd), torch.empty_like(eager)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fg.linear_epilogue(buf, Wq, Ws, F32, bias=bd, act="gelu", residual=Rd, Y=out)
        buf.copy_(Xd)
        graph.replay()
        assert torch.equal(eager, out)
    fg.check_device_status()


def test_callers_buffers(dev):
    """The quantizer's buffers given whole, in part or not at all; the codes
    and scales left in them are the quantizer's."""
    M, N, K = 70, 256, 640
    for fmt in (F32, UE8M0):
        X, Wq, Ws, b, R = make(dev, M, N, K, fmt, torch.float32, True, seed=4)
        kw = dict(bias=b.to(dev), act="relu", residual=R.to(dev))
        Xd = X.to(dev)
        ref = fg.linear_epilogue(Xd, Wq, Ws, fmt, **kw)
        Xq, Xs = fg.quant_act(Xd, fmt)
        ld = Xs.shape[1] + 32
        for q, s in ((1, 0), (0, 1), (1, 1)):
            bq = torch.empty_like(Xq) if q else None
            bs = torch.empty((K // 128, ld), dtype=Xs.dtype, device=dev) if s else None
            assert torch.equal(ref, fg.linear_epilogue(Xd, Wq, Ws, fmt, Xq=bq, Xs=bs, ld_s=ld, **kw))
            assert bq is None or torch.equal(bq, Xq)
            assert bs is None or torch.equal(bs[:, :M], Xs[:, :M])
    fg.check_device_status()


def test_empty(dev):
    Wq, Ws = fg.quant_weight(workloads.weights((256, 128), seed=1).to(dev), F32)
    assert fg.linear_epilogue(torch.empty(0, 128, dtype=torch.bfloat16, device=dev), Wq, Ws, F32).shape == (0, 256)
    fg.check_device_status()


@pytest.mark.parametrize("fmt", [F32, UE8M0])
def test_quantizing_inside_leaves_the_same_bits(dev, fmt):
    """Up to FUSED_QUANT_TOKENS tokens the kernel quantizes X itself: the same
    codes, scales, split and order of sums as from the quantizer's buffers, so
    the same bits; rows with NaN and infinities end as they do there, and the
    other rows are as if those were not among them."""
    for M in (1, 5, fg.FUSED_QUANT_TOKENS):
        X, Wq, Ws, b, R = make(dev, M, 384, 1152, fmt, torch.float32, True, seed=M)
        kw = dict(bias=b.to(dev), act="gelu_tanh", residual=R.to(dev))
        clean = fg.linear_epilogue(X.to(dev), Wq, Ws, fmt, **kw)
        X[0, 130], X[M // 2, 1000] = float("nan"), float("-inf")
        Xd = X.to(dev)
        Xq, Xs = fg.quant_act(Xd, fmt)
        got = fg.linear_epilogue(Xd, Wq, Ws, fmt, **kw)
        ref = fg.gemm_epilogue(Xq, Xs, Wq, Ws, fmt, **kw)
        assert got[0].isnan().all()
        for m in range(M):
            assert torch.equal(got[m].nan_to_num(1.5), ref[m].nan_to_num(1.5)) and torch.equal(got[m].isnan(), ref[m].isnan())
            if m not in (0, M // 2):
                assert torch.equal(got[m], clean[m])
    fg.check_device_status()


@pytest.mark.parametrize("fmt", [F32, UE8M0])
def test_offsets_past_32_bits(dev, fmt):
    """An output of more than 2^31 elements, added to in place: the rows on both
    sides of the border and the last ones."""
    M, N, K = 65800, 32768, 128
    X = workloads.activations((M, K), "normal", seed=1)
    Wq, Ws = fg.quant_weight(workloads.weights((N, K), seed=2).to(dev), fmt)
    b = torch.randn(N, generator=torch.Generator().manual_seed(3))
    Y = torch.full((M, N), 0.75, dtype=torch.bfloat16, device=dev)
    fg.linear_epilogue(X.to(dev), Wq, Ws, fmt, bias=b.to(dev), act="silu", residual=Y, Y=Y)
    fg.check_device_status()
    rows = np.array([0, 32767, 32768, 65535, 65536, 65537, M - 1])
    for r in rows:
        one = X[r:r + 1]
        y, tol = reference(one, Wq, Ws, fmt, b, "silu", torch.full((1, N), 0.75, dtype=torch.bfloat16))
        check(Y[int(r):int(r) + 1], y, tol, f"row {r}")
