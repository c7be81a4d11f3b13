"""Products whose waits may give up, in every kernel form: a status of 0 means a
complete result, a timeout is reported, and later calls are not touched."""

import pytest
import torch

import padding_free_packed_gb300 as pe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
TIMEOUT = 7

# 16, 32 and 64 rows a CTA without and with a split sum; pairs on whole and on shared
# tiles.
WAYS = [(5, 300, 500, BF16), (3, 512, 4000, FP32), (320, 1001, 1140, BF16),
        (300, 130, 20000, FP32), (1537, 768, 1152, FP32), (768, 768, 4500, BF16),
        (768, 768, 9001, BF16), (9000, 1152, 768, BF16), (9000, 1001, 768, FP32), (2304, 768, 20000, FP32),
        (2500, 999, 9001, BF16)]


def _product(m, n, k):
    gen = torch.Generator(device=DEV).manual_seed(531)
    a = torch.randn(m, k, generator=gen, device=DEV)
    b = torch.randn(n, k, generator=gen, device=DEV)
    return (*pe.pe_quantize_fp8(a), *pe.pe_quantize_fp8(b, 128))


@pytest.mark.parametrize("m,n,k,dtype", WAYS)
def test_a_wait_that_gives_up_is_reported(m, n, k, dtype):
    ops = _product(m, n, k)
    want = pe.pe_matmul_fp8(*ops, dtype=dtype)
    assert pe.pe_read_matmul_status() == 0
    previous = pe.pe_set_wait_limit_ns(1)
    try:
        pe.pe_matmul_fp8(*ops, dtype=dtype)
        assert pe.pe_read_matmul_status() == TIMEOUT
    finally:
        pe.pe_set_wait_limit_ns(previous)
    assert torch.equal(pe.pe_matmul_fp8(*ops, dtype=dtype), want)
    assert pe.pe_read_matmul_status() == 0


@pytest.mark.parametrize("limit_ns", [300, 1500, 4000, 20000])
@pytest.mark.parametrize("m,n,k,dtype", WAYS)
def test_status_0_means_a_complete_result(m, n, k, dtype, limit_ns):
    """Limits that some waits exceed; out holds NaN before each call, so that
    nothing of an earlier one can pass for a result."""
    ops = _product(m, n, k)
    want = pe.pe_matmul_fp8(*ops, dtype=dtype)
    out = torch.empty_like(want)
    assert pe.pe_read_matmul_status() == 0
    previous = pe.pe_set_wait_limit_ns(limit_ns)
    try:
        for _ in range(4):
            out.fill_(float("nan"))
            pe.pe_matmul_fp8(*ops, out=out)
            status = pe.pe_read_matmul_status()
            assert status in (0, TIMEOUT)
            assert status == TIMEOUT or torch.equal(out, want)
    finally:
        pe.pe_set_wait_limit_ns(previous)
    out.fill_(float("nan"))
    pe.pe_matmul_fp8(*ops, out=out)
    assert pe.pe_read_matmul_status() == 0 and torch.equal(out, want)
