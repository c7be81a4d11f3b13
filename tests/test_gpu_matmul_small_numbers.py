"""fp32 products of numbers near the ends of fp32's range, which the tensor cores get in bf16
parts: small ones keep all their bits."""

import pytest
import torch

import padding_free_packed_gb300 as pe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LAYOUTS = [(False, False), (False, True), (True, False), (True, True)]
# As they lie (m = 1 and 20 of plain layout), few rows, whole tiles, and slices.
SIZES = [(1, 300), (20, 300), (60, 640), (400, 1000), (5000, 777), (300, 9000)]


def _stored(x, transposed):
    x = x.t() if transposed else x
    view = torch.full((x.shape[0], x.shape[1] + 7 & -8), float("nan"), device=DEV)
    view = view[:, :x.shape[1]]
    return view.copy_(x)


def _numbers(gen, rows, cols, low, high):
    """24-bit numbers of either sign with exponents from low to high, in 64 bits."""
    bits = torch.randint(1 << 23, 1 << 24, (rows, cols), generator=gen, device=DEV).double()
    sign = torch.randint(0, 2, (rows, cols), generator=gen, device=DEV) * 2 - 1
    exponent = torch.randint(low - 23, high - 22, (rows, cols), generator=gen, device=DEV)
    return bits * sign * torch.pow(2.0, exponent.double())


def _picks(n, k, number, gen):
    """A matrix with one number in a row, and the columns where it stands."""
    at = torch.randperm(k, generator=gen, device=DEV)[:n]
    b = torch.zeros(n, k, device=DEV)
    b[torch.arange(n, device=DEV), at] = number
    return b, at


@pytest.mark.parametrize("swapped", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m,k", SIZES)
def test_small_numbers_times_a_large_one_come_back_exactly(m, k, layout, swapped):
    """2^-124 is the smallest number whose last bit, 2^-147, three parts hold."""
    gen = torch.Generator(device=DEV).manual_seed(72)
    x = _numbers(gen, m, k, -124, -100)
    pick, at = _picks(min(k, 640), k, 2.0 ** 100, gen)
    want = (x[:, at] * 2.0 ** 100).float()
    a, b = (pick, x.float()) if swapped else (x.float(), pick)
    got = pe.pe_matmul(_stored(a, layout[0]), _stored(b, layout[1]), a_transposed=layout[0],
                       b_transposed=layout[1])
    assert pe.pe_read_matmul_status() == 0
    assert torch.equal(got.t() if swapped else got, want)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m,k", SIZES)
def test_the_smallest_numbers_are_off_by_their_last_bits(m, k, layout):
    """Below 2^-124 three parts hold multiples of 2^-147, to within half of one: down to fp32's
    smallest number, 2^-149."""
    gen = torch.Generator(device=DEV).manual_seed(76)
    x = _numbers(gen, m, k, -126, -124)
    tiny = torch.randint(-(1 << 23), 1 << 23, (m, k), generator=gen, device=DEV).double()
    x = torch.where(torch.rand(m, k, generator=gen, device=DEV) < 0.5, x, tiny * 2.0 ** -149)
    x = x.float()
    pick, at = _picks(min(k, 640), k, 2.0 ** 100, gen)
    got = pe.pe_matmul(_stored(x, layout[0]), _stored(pick, layout[1]), a_transposed=layout[0],
                       b_transposed=layout[1])
    off = (got.double() * 2.0 ** -100 - x[:, at].double()).abs().max()
    assert float(off) <= 2.0 ** -148
