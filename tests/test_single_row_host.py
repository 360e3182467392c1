"""Operands of a single row in the binding of the epilogue GEMM, the router and
the expert layer (CPU only): the kernels read a row as contiguous, so a column
stride other than one is refused whatever the number of rows, and a single
row's own stride, which nothing reads, is not looked at."""
import pytest
import torch

import fine_grained_fp8_token_b200 as fg

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def rows(kind, C, dtype):
    """A [1, C] tensor whose elements do not lie side by side."""
    big = torch.zeros(max(C, 8), 2 * C, dtype=dtype)
    if kind == "column":
        return big[:C, 3:4].t()                              # strides (1, 2 C)
    if kind == "step":
        return big[:1, ::2]                                  # strides (2 C, 2)
    return torch.zeros(1, 1, dtype=dtype).expand(1, C)       # strides (1, 0), one element of storage


def calls(x, K):
    """The calls that take x ([1, K], bf16 or, for the router, any type) as an operand."""
    Wq, Ws = torch.zeros(K, K, dtype=U8), torch.zeros(K // 128, K // 128)
    W13q, W13s = torch.zeros(2, 2 * K, K, dtype=U8), torch.zeros(2, 2 * K // 128, K // 128)
    W2q, W2s = torch.zeros(2, K, K, dtype=U8), torch.zeros(2, K // 128, K // 128)
    X = torch.zeros(1, K, dtype=BF16)
    Xq, Xs = torch.zeros(1, K, dtype=U8), torch.zeros(K // 128, 4)
    ids, w = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2)
    moe = (W13q, W13s, W2q, W2s, 0)
    return {
        "linear X": lambda: fg.linear_epilogue(x, Wq, Ws, 0),
        "linear residual": lambda: fg.linear_epilogue(X, Wq, Ws, 0, residual=x),
        "gemm residual": lambda: fg.gemm_epilogue(Xq, Xs, Wq, Ws, 0, residual=x),
        "moe X": lambda: fg.moe_decode(x, ids, w, *moe),
        "moe residual": lambda: fg.moe_decode(X, ids, w, *moe, residual=x),
        "logits": lambda: fg.route_topk(x, 2),
        "logits fp32": lambda: fg.route_topk(x.float() if x.stride(1) == 1 else rows_like(x), 2),
    }


def rows_like(x):
    y = torch.empty_strided(x.shape, x.stride(), dtype=F32)
    return y


CALLS = ["linear X", "linear residual", "gemm residual", "moe X", "moe residual", "logits", "logits fp32"]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kind", ["column", "step", "expand"])
def test_a_single_row_that_is_not_contiguous_is_refused(kind, call):
    K = 128
    x = rows(kind, K, BF16)
    assert x.shape == (1, K) and x.stride(1) != 1
    with pytest.raises(fg.FGFP8Error, match="unit stride"):
        calls(x, K)[call]()


@pytest.mark.parametrize("call", CALLS)
def test_the_row_stride_of_a_single_row_is_not_looked_at(call):
    """A row of a wider buffer, and one with a row stride of zero or of an odd
    number: past this check, they reach the next one (no GPU tensor)."""
    K = 128
    wide = torch.zeros(4, K + 40, dtype=BF16)
    for x in (wide[2:3, 8:8 + K], torch.zeros(K, dtype=BF16).expand(1, K), torch.zeros(K, dtype=BF16).as_strided((1, K), (77, 1))):
        assert x.stride(1) == 1
        with pytest.raises(fg.FGFP8Error, match="CUDA device"):
            calls(x, K)[call]()


def test_no_rows_and_one_column():
    """Nothing is read of an empty operand, and a single column's stride says nothing."""
    K = 128
    Wq, Ws = torch.zeros(K, K, dtype=U8), torch.zeros(1, 1)
    for x in (torch.zeros(0, 2 * K, dtype=BF16)[:, ::2], torch.zeros(4, K, dtype=BF16)[:0]):
        with pytest.raises(fg.FGFP8Error, match="CUDA device"):
            fg.linear_epilogue(x, Wq, Ws, 0)
    for z in (torch.zeros(1, 5)[:, ::5], torch.zeros(3, 5)[:, 2:3]):
        with pytest.raises(fg.FGFP8Error, match="CUDA device"):
            fg.route_topk(z, 1)
