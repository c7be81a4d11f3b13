"""fp32 products by parts on the tensor cores: every part of either operand, and the products of
the parts, arrive exactly, up to fp32's largest number."""

import pytest
import torch

import padding_free_packed_gb300 as pe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FP32 = torch.float32
LAYOUTS = [(False, False), (False, True), (True, False), (True, True)]
# Few rows (as they lie where the layout is plain), whole tiles, and slices of a long sum.
SIZES = [(1, 300, 300), (20, 300, 300), (60, 640, 640), (400, 1000, 1000), (5000, 777, 777),
         (2100, 2100, 2100), (300, 300, 9000)]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _stored(x, transposed):
    x = x.t() if transposed else x
    view = torch.full((x.shape[0], x.shape[1] + 7 & -8), float("nan"), device=DEV)
    view = view[:, :x.shape[1]]
    return view.copy_(x)


def _product(a, b, layout):
    got = pe.pe_matmul(_stored(a, layout[0]), _stored(b, layout[1]), a_transposed=layout[0],
                       b_transposed=layout[1])
    assert pe.pe_read_matmul_status() == 0
    return got


def _picks(rows, k, gen, values=1.0):
    """A matrix with one number in a row, and the columns where it stands."""
    at = torch.randint(0, k, (rows,), generator=gen, device=DEV)
    x = torch.zeros(rows, k, device=DEV)
    x[torch.arange(rows, device=DEV), at] = values
    return x, at


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_a_picks_columns_of_b_exactly(m, n, k, layout):
    """24-bit numbers in b, far from one another in size."""
    gen = _gen(73)
    b = torch.randn(n, k, generator=gen, device=DEV)
    b *= torch.exp(4 * torch.randn(n, k, generator=gen, device=DEV))
    a, at = _picks(m, k, gen)
    assert torch.equal(_product(a, b, layout), b[:, at].t())


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_products_of_middle_parts_are_exact(m, n, k, layout):
    """(1 + i / 2^12) (1 + j / 2^10) with i below 16 and j from 1 to 3: both are 1 and a middle
    part, and the product, with the middle parts' i j / 2^22, fits 24 bits."""
    gen = _gen(74)
    b = 1 + torch.randint(0, 16, (n, k), generator=gen, device=DEV).float() / 4096
    j = torch.randint(1, 4, (m,), generator=gen, device=DEV).float()
    a, at = _picks(m, k, gen, 1 + j / 1024)
    want = (b[:, at].t().double() * (1 + j / 1024).double()[:, None]).float()
    assert torch.equal(_product(a, b, layout), want)


@pytest.mark.parametrize("swapped", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m,k", [(1, 96), (80, 96), (700, 200), (5000, 640), (300, 9000)])
def test_numbers_up_to_the_largest_come_back_exactly(m, k, layout, swapped):
    """Numbers that rounding to bf16 would make infinite are cut off instead."""
    gen = _gen(75)
    some = torch.tensor([3.4028234663852886e38, -3.4e38, 3.3961e38, 1.0, -2.0 ** -60, 1.5e38],
                        device=DEV)
    x = some[torch.randint(0, 6, (m, k), generator=gen, device=DEV)]
    pick, at = _picks(min(k, 640), k, gen)
    got = _product(pick, x, layout) if swapped else _product(x, pick, layout)
    assert torch.equal(got.t() if swapped else got, x[:, at])
