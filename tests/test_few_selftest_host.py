"""Refusals of the few-token kernels' self-tests on the host (CPU only)."""
import pytest
import torch

import fine_grained_fp8_token_b200 as fg

INVALID, SHAPE, CUDA = 1, 2, 5
A = 1 << 20          # a fake, 256-byte aligned "device" address; never dereferenced on these paths


def few(M=4, N=512, K=1024, fmt=0, withhold=1, Xq=A):
    return fg.fgfp8_selftest_few_timeout(Xq, A, 64, A, A, A, M, N, K, fmt, withhold, None)


def moe(T=4, E=4, K=1024, kernel=0, withhold=1, ws_bytes=1 << 30):
    return fg.fgfp8_selftest_moe_timeout(A, K, A, A, A, A, A, A, A, A, ws_bytes, T, 2, E, K, 256, 0, kernel, withhold, None)


def test_refusals():
    assert few(withhold=8) == few(withhold=-1) == INVALID
    assert few(M=65) == few(M=0) == SHAPE
    assert few(N=100) == few(K=1000) == SHAPE
    assert few(fmt=2) == few(Xq=None) == INVALID
    assert moe(kernel=2) == moe(kernel=-1) == moe(withhold=-1) == moe(withhold=1 << 31) == INVALID
    assert moe(T=65) == moe(E=513) == moe(ws_bytes=16) == SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the behaviour without a GPU")
def test_no_cpu_path():
    assert few() == moe() == moe(kernel=1) == CUDA
