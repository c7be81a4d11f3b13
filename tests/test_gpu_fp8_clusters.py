"""Products whose CTAs read one another's shared memory or signal one another's
barriers: every width of the last column tile, and many short launches in a row."""

import pytest
import torch

import fp8_reference as ref
import padding_free_packed_gb300 as pe
from test_gpu_fp8 import _gen, _operands

pytestmark = pytest.mark.gpu
FP32 = torch.float32


@pytest.mark.parametrize("m", [3, 20, 60])
@pytest.mark.parametrize("n", [1, 2, 5, 31, 66, 127, 130, 135, 253])
def test_split_sums_with_a_ragged_last_column_tile(m, n):
    """Lanes whose columns lie past n leave the join early; the CTAs stay until the
    whole cluster has read their sums."""
    a, sa, b, sb = _operands(_gen(541), m, n, 6000, ints=True)
    want, _ = ref.matmul(a, sa, b, sb)
    for _ in range(20):
        assert torch.equal(pe.pe_matmul_fp8(a, sa, b, sb, dtype=FP32).double(), want)
    assert pe.pe_read_matmul_status() == 0


@pytest.mark.parametrize("m,n,k", [(9000, 1152, 128), (40000, 256, 130), (2304, 768, 20000)])
def test_many_launches_of_pairs_in_a_row(m, n, k):
    """Each launch reuses the shared memory that the one before signalled into."""
    a, sa, b, sb = _operands(_gen(542), m, n, k, ints=True)
    want, _ = ref.matmul(a, sa, b, sb)
    outs = [torch.empty(m, n, dtype=FP32, device=a.device) for _ in range(4)]
    for i in range(200):
        pe.pe_matmul_fp8(a, sa, b, sb, out=outs[i % 4])
    for out in outs:
        assert torch.equal(out.double(), want)
    assert pe.pe_read_matmul_status() == 0
