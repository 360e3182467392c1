"""Refusals of the epilogue GEMM, the router and the few-token expert layer on
the host (CPU only): every bad argument is an error before any launch, and a
good call without a GPU is a CUDA error, never a CPU result."""
import ctypes

import pytest
import torch

import fine_grained_fp8_token_b200 as fg

OK, INVALID, SHAPE, ALIGN, UNSUP, CUDA = 0, 1, 2, 3, 4, 5
A = 1 << 20          # a fake, 256-byte aligned "device" address; never dereferenced on these paths


def linear(**kw):
    a = dict(X=A << 2, ldx=256, Xq=A, Xs=A, ld_s=4, Wq=A, Ws=A, Y=A, M=4, N=128, K=256, fmt=0, bias=None, bias_type=0, act=0,
             residual=None, ld_r=0)
    a.update(kw)
    return fg.fgfp8_linear_epilogue(*a.values(), None)


def gemm(**kw):
    a = dict(Xq=A, Xs=A, ld_s=4, Wq=A, Ws=A, Y=A, M=4, N=128, K=256, fmt=0, bias=None, bias_type=0, act=0, residual=None,
             ld_r=0)
    a.update(kw)
    return fg.fgfp8_gemm_epilogue(*a.values(), None)


EPILOGUE = [(dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(bias_type=2), INVALID), (dict(bias=A + 2), ALIGN),
            (dict(residual=A << 2, ld_r=120), SHAPE), (dict(residual=A, ld_r=132), ALIGN), (dict(residual=A + 8, ld_r=128), ALIGN),
            (dict(Wq=None), INVALID), (dict(Y=None), INVALID), (dict(Y=A + 4), ALIGN), (dict(Ws=A + 2), ALIGN),
            (dict(fmt=2), INVALID), (dict(N=100), SHAPE), (dict(N=0), SHAPE), (dict(K=200, ldx=200), SHAPE),
            (dict(K=0), SHAPE), (dict(N=-128), INVALID)]


@pytest.mark.parametrize("M", [4, 40, 400])
@pytest.mark.parametrize("bad,code", EPILOGUE)
def test_epilogue_refusals(M, bad, code):
    kw = dict(M=M, ld_s=400, **bad)
    assert linear(**kw) == code, bad
    kw.pop("ldx", None)
    assert gemm(**kw) == code, bad
    assert fg.fgfp8_last_error_string() != ""


def test_overlaps_are_refused():
    far = A + (1 << 24)
    for M in (1, 4, 40, 400):
        kw = dict(M=M, ld_s=400, X=far, Xq=far, Xs=far)
        # the residual may be Y itself, row by row, and nothing else that meets it
        assert linear(**kw, residual=A, ld_r=128) == gemm(M=M, ld_s=400, residual=A, ld_r=128)
        if not torch.cuda.is_available():
            assert linear(**kw, residual=A, ld_r=128) == CUDA
            assert linear(**kw, residual=A + 2 * M * 128, ld_r=128) == CUDA
        if M > 1:
            assert linear(**kw, residual=A, ld_r=256) == INVALID
            assert gemm(M=M, ld_s=400, residual=A + 256, ld_r=128) == INVALID
        assert linear(**kw, residual=A + 16, ld_r=128) == INVALID
        assert linear(M=M, ld_s=400, X=A) == INVALID                       # X is Y
        assert linear(M=M, ld_s=400, X=A - 2 * M * 256 + 32, Y=A) == INVALID
    assert moe(X=far, residual=A + 512, ld_r=256) == INVALID


def test_linear_epilogue_operand_refusals():
    for M in (4, 40):
        assert linear(M=M, ld_s=64, ldx=128) == SHAPE
        assert linear(M=M, ld_s=64, ldx=257) == ALIGN
        assert linear(M=M, ld_s=64, X=None) == INVALID
        assert linear(M=M, ld_s=64, X=A + 2) == ALIGN
    assert linear(M=40, ld_s=64, Xq=None) == INVALID
    assert linear(M=40, ld_s=64, Xs=None) == INVALID
    assert linear(M=40, ld_s=32) == SHAPE
    assert linear(M=-1) == INVALID
    assert linear(M=0) == OK and gemm(M=0) == OK


def route(**kw):
    a = dict(logits=A, ltype=1, ld=64, bias=None, T=4, E=64, topk=4, score=0, n_group=1, topk_group=1, renorm=1, scale=1.0,
             ids=A, weights=A)
    a.update(kw)
    return fg.fgfp8_route_topk(*a.values(), None)


@pytest.mark.parametrize("bad,code", [
    (dict(ltype=2), INVALID), (dict(score=2), INVALID), (dict(renorm=2), INVALID), (dict(T=-1), INVALID),
    (dict(E=0), SHAPE), (dict(E=513, ld=513), SHAPE), (dict(ld=63), SHAPE), (dict(topk=0), SHAPE), (dict(topk=17), SHAPE),
    (dict(E=2, topk=3), SHAPE), (dict(n_group=0), SHAPE), (dict(n_group=3), SHAPE), (dict(n_group=64), SHAPE),
    (dict(n_group=4, topk_group=5), SHAPE), (dict(topk_group=0), SHAPE), (dict(bias=A), UNSUP), (dict(logits=None), INVALID),
    (dict(ids=None), INVALID), (dict(weights=None), INVALID), (dict(logits=A + 2), ALIGN), (dict(ltype=0, logits=A + 1), ALIGN),
    (dict(ids=A + 2), ALIGN), (dict(score=1, bias=A + 1), ALIGN), (dict(T=1 << 31), SHAPE)])
def test_route_refusals(bad, code):
    assert route(**bad) == code, bad


def moe(**kw):
    a = dict(X=A, ldx=256, ids=A, weights=A, W13q=A, W13s=A, W2q=A, W2s=A, residual=None, ld_r=0, Y=A, ws=A, ws_bytes=1 << 30,
             T=4, topk=2, E=8, K=256, I=128, fmt=0)
    a.update(kw)
    return fg.fgfp8_moe_decode(*a.values(), None)


@pytest.mark.parametrize("bad,code", [
    (dict(T=65), SHAPE), (dict(T=-1), INVALID), (dict(topk=0), SHAPE), (dict(topk=17), SHAPE), (dict(E=0), SHAPE),
    (dict(E=513), SHAPE), (dict(K=200), SHAPE), (dict(K=0), SHAPE), (dict(I=0), SHAPE), (dict(I=64), SHAPE), (dict(ldx=128), SHAPE),
    (dict(ldx=260), ALIGN), (dict(fmt=3), INVALID), (dict(ws_bytes=100), SHAPE), (dict(ws=A + 16), ALIGN), (dict(ws=None), INVALID),
    (dict(Y=None), INVALID), (dict(ids=None), INVALID), (dict(ids=A + 1), ALIGN), (dict(weights=A + 2), ALIGN),
    (dict(W2q=A + 8), ALIGN), (dict(W13s=A + 1), ALIGN), (dict(residual=A, ld_r=128), SHAPE), (dict(residual=A, ld_r=257), ALIGN),
    (dict(E=512, I=1 << 21), SHAPE), (dict(E=512, K=1 << 22, ldx=1 << 22), SHAPE)])
def test_moe_refusals(bad, code):
    assert moe(**bad) == code, bad


def test_moe_workspace_size():
    n = ctypes.c_int64(-5)
    f = fg.fgfp8_moe_workspace_bytes
    # codes of H, then its scales, each from a 256-byte boundary
    assert f(3, 2, 256, 128, ctypes.byref(n)) == OK and n.value == 768 + 256
    # above 16 tokens the codes of X and its scales too
    assert f(17, 1, 256, 128, ctypes.byref(n)) == OK and n.value == 2304 + 256 + 4352 + 32 * 2 * 4
    assert fg.moe_workspace_bytes(0, 1, 128, 128) == 0
    assert f(65, 2, 256, 128, ctypes.byref(n)) == SHAPE
    assert f(3, 2, 256, 100, ctypes.byref(n)) == SHAPE
    assert f(3, 2, 100, 128, ctypes.byref(n)) == SHAPE
    assert f(3, 2, 256, 128, None) == INVALID
    need = fg.moe_workspace_bytes(4, 2, 256, 128)
    assert moe(ws_bytes=need - 1) == SHAPE
    assert moe(T=0, ws=None, ws_bytes=0, X=None) == OK


def test_no_cpu_path():
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    assert linear() == CUDA and gemm() == CUDA and route() == CUDA and moe() == CUDA
    assert linear(M=40, ld_s=64) == CUDA


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_wrong_tensors():
    """The tensor helpers check types, shapes, layouts and devices before any
    address is taken."""
    Wq, Ws, X = cpu(256, 128, dtype=torch.uint8), cpu(2, 1, dtype=torch.float32), cpu(4, 128)

    def bad(f, *a, match=None, **kw):
        with pytest.raises(fg.FGFP8Error, match=match):
            f(*a, **kw)
    bad(fg.linear_epilogue, X, Wq, Ws, 0, match="CUDA device")
    bad(fg.linear_epilogue, X.float(), Wq, Ws, 0, match="X must be")
    bad(fg.linear_epilogue, cpu(4, 256)[:, ::2], Wq, Ws, 0, match="unit stride")
    bad(fg.linear_epilogue, cpu(4, 256), Wq, Ws, 0, match="columns")
    bad(fg.linear_epilogue, X, Wq.float(), Ws, 0, match="Wq must be")
    bad(fg.linear_epilogue, X, Wq, Ws.to(torch.uint8), 0, match="Ws must be")
    bad(fg.linear_epilogue, X, Wq, Ws, 1, match="Ws must be")
    bad(fg.linear_epilogue, X, Wq, Ws, 7, match="fmt")
    bad(fg.linear_epilogue, X, Wq, Ws, 0, bias=cpu(128), match="bias must be")
    bad(fg.linear_epilogue, X, Wq, Ws, 0, act="tanh", match="act must be")
    bad(fg.linear_epilogue, X, Wq, Ws, 0, residual=cpu(4, 128), match="residual must be")
    bad(fg.linear_epilogue, X, Wq, Ws, 0, Y=cpu(4, 128), match="Y must be")
    bad(fg.gemm_epilogue, cpu(4, 128, dtype=torch.uint8), cpu(1, 4, dtype=torch.float32), Wq, Ws, 0, match="CUDA device")
    bad(fg.gemm_epilogue, X, cpu(1, 4, dtype=torch.float32), Wq, Ws, 0, match="Xq must be")
    z = cpu(4, 32, dtype=torch.float32)
    bad(fg.route_topk, z, 4, match="CUDA device")
    bad(fg.route_topk, z.double(), 4, match="logits")
    bad(fg.route_topk, z, 4, score="max", match="score")
    bad(fg.route_topk, z, 4, score="sigmoid", bias=cpu(31, dtype=torch.float32), match="bias")
    bad(fg.route_topk, z, 4, ids=cpu(4, 3, dtype=torch.int32), match="ids")
    bad(fg.route_topk, z, 0, match="topk")
    W13q, W13s = cpu(2, 256, 128, dtype=torch.uint8), cpu(2, 2, 1, dtype=torch.float32)
    W2q, W2s = cpu(2, 128, 128, dtype=torch.uint8), cpu(2, 1, 1, dtype=torch.float32)
    ids, w = cpu(4, 2, dtype=torch.int32), cpu(4, 2, dtype=torch.float32)
    bad(fg.moe_decode, X, ids, w, W13q, W13s, W2q, W2s, 0, match="CUDA device")
    bad(fg.moe_decode, X, ids.long(), w, W13q, W13s, W2q, W2s, 0, match="ids must be")
    bad(fg.moe_decode, X, ids, w.bfloat16(), W13q, W13s, W2q, W2s, 0, match="weights must be")
    bad(fg.moe_decode, X, ids, w, W13q[:, :128], W13s, W2q, W2s, 0)
    bad(fg.moe_decode, X, ids, w, W2q, W2s, W2q, W2s, 0, match="2I")
    bad(fg.moe_decode, X, ids, w, W13q, W13s, W2q, W2s, 0, residual=cpu(3, 128), match="residual")
