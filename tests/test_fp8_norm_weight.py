"""A norm's weight comes in the rows' dtype: rounding it is the caller's choice."""

import pytest
import torch

import padding_free_packed_gb300 as pe
from padding_free_packed_gb300 import binding

BF16, FP32 = torch.bfloat16, torch.float32


def test_a_weight_of_another_type_is_refused():
    for rows, weight in ((BF16, FP32), (FP32, BF16), (BF16, torch.float16)):
        with pytest.raises(ValueError, match="weight must be"):
            binding._norm_weight(torch.ones(64, dtype=weight), torch.ones(4, 64, dtype=rows), 64)
    with pytest.raises(TypeError, match="unsupported dtype"):
        binding._norm_weight(torch.ones(64), torch.ones(4, 64, dtype=torch.float16), 64)


@pytest.mark.gpu
def test_no_norm_rounds_its_weight():
    """1 + 2^-10 is 1 in bf16."""
    x = torch.ones(4, 64, dtype=BF16, device="cuda:0")
    w = torch.full((64,), 1 + 2.0 ** -10, device="cuda:0")
    for call in (lambda: pe.pe_rmsnorm(x, w), lambda: pe.pe_rmsnorm_fp8(x, w),
                 lambda: pe.pe_rmsnorm_bwd(x, x, w)):
        with pytest.raises(ValueError, match="weight must be"):
            call()
    assert torch.equal(pe.pe_rmsnorm(x, w.to(BF16)), pe.pe_rmsnorm(x, torch.ones_like(x[0])))
