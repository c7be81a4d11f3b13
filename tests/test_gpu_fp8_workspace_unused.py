"""An 8-bit product that needs no workspace does not look at the caller's."""

import pytest
import torch

import padding_free_packed_gb300 as pe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("m,n,k", [(5, 300, 256), (3000, 768, 768)])
def test_any_workspace_is_taken_where_none_is_needed(m, n, k):
    gen = torch.Generator(device=DEV).manual_seed(552)
    a, sa = pe.pe_quantize_fp8(torch.randn(m, k, generator=gen, device=DEV))
    b, sb = pe.pe_quantize_fp8(torch.randn(n, k, generator=gen, device=DEV), 128)
    assert pe.load_library().pe_matmul_fp8_workspace_size(m, n, k) == 0
    want = pe.pe_matmul_fp8(a, sa, b, sb)
    store = torch.full((64, 2), 7, dtype=torch.uint8, device=DEV)
    for ws in (store, store[:, 0], store[:0], store.cpu()):
        assert torch.equal(pe.pe_matmul_fp8(a, sa, b, sb, workspace=ws), want)
    assert bool((store == 7).all())
