"""A caller's workspace is checked before a kernel writes there."""

import pytest
import torch

import padding_free_packed_gb300 as pe
from padding_free_packed_gb300 import binding

CPU = torch.device("cpu")


def test_only_contiguous_memory_of_the_device_is_a_workspace():
    store = torch.empty(64, dtype=torch.uint8)
    assert binding._workspace_for(store, 64, CPU) == (store, 64)
    words = torch.empty(16, dtype=torch.float32)
    assert binding._workspace_for(words, 64, CPU) == (words, 64)
    own, size = binding._workspace_for(None, 100, CPU)
    assert size >= 100 and own.numel() == size
    for bad in (store[::2], torch.empty(1, dtype=torch.uint8).expand(1 << 20),
                torch.empty(4, 8, dtype=torch.uint8).t()):
        with pytest.raises(ValueError, match="workspace"):
            binding._workspace_for(bad, 8, CPU)
    with pytest.raises(ValueError, match="cuda:0"):
        binding._workspace_for(store, 64, torch.device("cuda", 0))


@pytest.mark.gpu
def test_calls_refuse_other_workspaces():
    """Memory of the host, and views whose elements are not adjacent."""
    x, w = torch.ones(40, 64, device="cuda:0"), torch.ones(64, device="cuda:0")
    need = pe.load_library().pe_rmsnorm_bwd_workspace_size(64)
    a, sa = pe.pe_quantize_fp8(torch.ones(2304, 9000, device="cuda:0"))
    b, sb = pe.pe_quantize_fp8(torch.ones(768, 9000, device="cuda:0"), 128)
    more = max(need, pe.load_library().pe_matmul_fp8_workspace_size(2304, 768, 9000))
    good = torch.empty(more, dtype=torch.uint8, device="cuda:0")
    for bad in (good.cpu(), good[:1].expand(more), torch.empty(more, 2, dtype=torch.uint8,
                                                               device="cuda:0")[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            pe.pe_rmsnorm_bwd(x, x, w, workspace=bad)
        with pytest.raises(ValueError, match="workspace"):
            pe.pe_matmul_fp8(a, sa, b, sb, workspace=bad)
    want = pe.pe_matmul_fp8(a, sa, b, sb)
    words = torch.empty(more // 4, dtype=torch.float32, device="cuda:0")
    assert torch.equal(pe.pe_matmul_fp8(a, sa, b, sb, workspace=words), want)


@pytest.mark.gpu
@pytest.mark.parametrize("n,c,dtype", [(1, 768, torch.bfloat16), (300, 333, torch.float32),
                                       (5000, 768, torch.bfloat16)])
def test_calls_in_turn_through_one_workspace(n, c, dtype):
    """The second kernel of a call sums what the first left in the workspace, never what
    the call before did."""
    gen = torch.Generator(device="cuda:0").manual_seed(551)
    sets = [[torch.randn(n, c, generator=gen, device="cuda:0").to(dtype) for _ in range(2)]
            for _ in range(2)]
    w = torch.ones(c, device="cuda:0", dtype=dtype)
    want = [pe.pe_rmsnorm_bwd(*s, w) for s in sets]
    ws = torch.full((pe.load_library().pe_rmsnorm_bwd_workspace_size(c),), 0xFF,
                    dtype=torch.uint8, device="cuda:0")
    got = [pe.pe_rmsnorm_bwd(*sets[i % 2], w, workspace=ws) for i in range(200)]
    for i, one in enumerate(got):
        assert torch.equal(one[0], want[i % 2][0]) and torch.equal(one[1], want[i % 2][1])
