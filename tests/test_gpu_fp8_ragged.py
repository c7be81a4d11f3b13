"""The pair kernel's ragged edges against 64-bit references: an odd number of
128-column blocks (the second half of the last tile is absent), rows of out that
start anywhere, and shared tiles whose parts end inside a tile."""

import pytest
import torch

import fp8_reference as ref
import padding_free_packed_gb300 as pe
from test_gpu_fp8 import _close, _fenced, _gen, _operands, _outside_untouched

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32

# (m, n, k, whether pairs share tiles: only that way needs a workspace).
SHAPES = [(9000, 1152, 768, False), (9000, 1000, 768, False), (9000, 1001, 768, False),
          (2305, 1144, 20001, True), (2500, 999, 9001, True), (2304, 768, 32299, True)]


def _takes_the_way(m, n, k, shared):
    assert (pe.load_library().pe_matmul_fp8_workspace_size(m, n, k) > 0) == shared


@pytest.mark.parametrize("m,n,k,shared", SHAPES)
def test_small_whole_numbers_are_exact(m, n, k, shared):
    """Operands -1, 0, 1 and scales 1/2, 1, 2: partial sums are multiples of 1/4
    below 2^20, which fp32 holds."""
    _takes_the_way(m, n, k, shared)
    a, sa, b, sb = _operands(_gen(521), m, n, k, ints=True)
    want, _ = ref.matmul(a, sa, b, sb)
    for dtype in (FP32, BF16):
        store, out = _fenced(m, n, dtype, 0x77)
        pe.pe_matmul_fp8(a, sa, b, sb, out=out)
        assert torch.equal(out, want.float().to(dtype))
        _outside_untouched(store, m, n, dtype, 0x77)
    assert pe.pe_read_matmul_status() == 0


@pytest.mark.parametrize("m,n,k,shared", SHAPES)
def test_real_values(m, n, k, shared):
    _takes_the_way(m, n, k, shared)
    a, sa, b, sb = _operands(_gen(522), m, n, k)
    want, size = ref.matmul(a, sa, b, sb)
    for dtype in (FP32, BF16):
        _close(pe.pe_matmul_fp8(a, sa, b, sb, dtype=dtype), want, ref.matmul_rel(k), dtype,
               f"{m} x {n} x {k} {dtype}", size)
