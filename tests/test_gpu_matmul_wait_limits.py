"""16- and 32-bit products whose waits may give up, in every kernel form: a status of 0 means
a complete result, a timeout is reported, and later calls are not touched."""

import pytest
import torch

import padding_free_packed_gb300 as pe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
TIMEOUT = 7

# (m, n, k, type, activation, residual, pre): few rows without and with a split sum, whole
# tiles and runs of blocks, boxes by TMA and element by element.
WAYS = [(5, 300, 512, BF16, "none", True, False), (3, 512, 4000, BF16, "geglu", False, True),
        (320, 1001, 1140, BF16, "gelu", False, False), (300, 136, 20000, FP32, "none", True, False),
        (9000, 1152, 768, BF16, "none", True, False), (9000, 1152, 768, BF16, "geglu", True, True),
        (9000, 1001, 256, FP32, "relu", True, False), (9000, 1152, 256, FP32, "none", True, False),
        (2304, 768, 20000, BF16, "none", True, False), (2500, 999, 9008, BF16, "gelu", False, True)]


def _call(way):
    m, n, k, dtype, act, residual, pre = way
    gen = torch.Generator(device=DEV).manual_seed(81)
    mk = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(dtype)  # noqa: E731
    a, b, bias = mk(m, k + 7 & -8)[:, :k], mk(n, k + 7 & -8)[:, :k], mk(n if act != "geglu" or
                                                                       n % 2 == 0 else n - 1)
    wide = n // 2 if act == "geglu" else n
    r = mk(m, wide) if residual else None
    out = torch.empty(m, wide, dtype=dtype, device=DEV)
    z = torch.empty(m, n, dtype=dtype, device=DEV) if pre else None

    def call():
        out.fill_(float("nan"))
        if z is not None:
            z.fill_(float("nan"))
        pe.pe_matmul(a, b, bias=bias, activation=act, residual=r, out=out, pre=z)
        return [out] if z is None else [out, z]

    return call


@pytest.mark.parametrize("way", WAYS)
def test_a_wait_that_gives_up_is_reported(way):
    call = _call(way)
    want = [t.clone() for t in call()]
    assert pe.pe_read_matmul_status() == 0
    previous = pe.pe_set_wait_limit_ns(1)
    try:
        call()
        assert pe.pe_read_matmul_status() == TIMEOUT
    finally:
        pe.pe_set_wait_limit_ns(previous)
    assert all(torch.equal(g, w) for g, w in zip(call(), want))
    assert pe.pe_read_matmul_status() == 0


@pytest.mark.parametrize("limit_ns", [300, 1500, 4000, 20000])
@pytest.mark.parametrize("way", WAYS)
def test_status_0_means_a_complete_result(way, limit_ns):
    """Limits that some waits exceed; the outputs hold NaN before each call, so that nothing
    of an earlier one can pass for a result."""
    call = _call(way)
    want = [t.clone() for t in call()]
    assert pe.pe_read_matmul_status() == 0
    previous = pe.pe_set_wait_limit_ns(limit_ns)
    try:
        for _ in range(4):
            got = call()
            status = pe.pe_read_matmul_status()
            assert status in (0, TIMEOUT)
            assert status == TIMEOUT or all(torch.equal(g, w) for g, w in zip(got, want))
    finally:
        pe.pe_set_wait_limit_ns(previous)
    assert all(torch.equal(g, w) for g, w in zip(call(), want))
    assert pe.pe_read_matmul_status() == 0
