"""Long sums of the 16- and 32-bit matrix product: no chain of additions in the tensor cores,
which cut a sum off at its last bit every 16 products, is as long as k."""

import pytest
import torch

import padding_free_packed_gb300 as pe
import tail_reference as ref
from tail_reference import U
from test_gpu_matmul import _check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
PLAIN, BOTH = (False, False), (True, True)


def test_bf16_results_of_numbers_of_one_sign():
    """The longest chain is 128 blocks of 64 or, past that, 8 blocks, whose sums are added in
    fp32: 32 steps of 16 products, 17 numbers each of which loses at most 2^-23 of the sum, and
    an addition for every 512 numbers. Each row of b has a size of its own, so that the results
    lie everywhere between two bf16 numbers."""
    m, n, k, piece = 1024, 4864, 1 << 19, 1 << 15
    gen = torch.Generator(device=DEV).manual_seed(71)
    a = torch.empty(m, k, dtype=BF16, device=DEV).uniform_(0.5, 1, generator=gen)
    b = torch.empty(n, k, dtype=BF16, device=DEV).uniform_(0.5, 1, generator=gen)
    b.mul_((1 + torch.rand(n, 1, generator=gen, device=DEV)).bfloat16())
    got = pe.pe_matmul(a, b)
    assert pe.pe_read_matmul_status() == 0
    rows = [0, 131, 777, 1023]
    want = torch.zeros(len(rows), n, dtype=torch.float64, device=DEV)
    for x in range(0, k, piece):
        want += a[rows, x:x + piece].double() @ b[:, x:x + piece].double().t()
    bound = (34 * 32 + k // 512) * U * want
    ref.assert_within(got[rows], want, ref.rounded(bound, want, BF16), "long sums")


# (m, n, k, type of the operands, layout, blocks of 64 in a chain, additions that round): few
# rows with and without a split sum, whole tiles by TMA and to rows that start anywhere, slices.
CHAINS = [(3, 512, 4000, BF16, PLAIN, 4, 10), (320, 300, 12000, BF16, PLAIN, 4, 10),
          (100, 1000, 2000, FP32, PLAIN, 4, 10), (5, 640, 3000, FP32, (False, True), 4, 10),
          (9000, 1152, 4096, BF16, PLAIN, 8, 2), (9000, 1001, 2049, BF16, (False, True), 8, 2),
          (9000, 1152, 2048, FP32, PLAIN, 8, 2), (2304, 768, 32299, BF16, BOTH, 4, 18),
          (2304, 768, 20000, FP32, BOTH, 4, 18), (300, 136, 70000, BF16, BOTH, 4, 18)]


@pytest.mark.parametrize("at", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("m,n,k,dtype,layout,blocks,roundings", CHAINS)
def test_small_numbers_beside_a_one_are_kept_outside_its_chain(m, n, k, dtype, layout, blocks,
                                                               roundings, at):
    """One product of 1 and otherwise products of 2^-28, 16 of which are 2^-24: too little to
    be added to a 1. Sums without the 1 are exact, so at most its own chain is lost, and half a
    step of a number below 2 where a sum that is not whole chains is added to the 1: once or
    twice in its slice, and for each of the other slices (8 of few rows, 16 of tiles)."""
    one = min(k - 1, int(at * k))

    def operand(size, transposed):
        rows, cols = (k, size) if transposed else (size, k)
        x = torch.full((rows, cols + 7 & -8), 2.0 ** -14, dtype=dtype, device=DEV)[:, :cols]
        (x[one] if transposed else x[:, one]).fill_(1)
        return x

    a, b = operand(m, layout[0]), operand(n, layout[1])
    got = pe.pe_matmul(a, b, dtype=FP32, a_transposed=layout[0], b_transposed=layout[1])
    want = 1 + (k - 1) * 2.0 ** -28
    assert 1 < want < 2
    bound = blocks * 64 * 2.0 ** -28 + roundings * U
    err = float((got.double() - want).abs().max())
    assert err <= bound, f"off by {err:.2e}, at most {bound:.2e}"


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "geglu"])
@pytest.mark.parametrize("m,n,k,layout", [(2300, 2048, 9000, PLAIN), (2300, 2046, 8200, (True, False))])
def test_epilogue_of_long_sums_to_bf16(m, n, k, layout, act):
    """Whole tiles of more than 128 blocks: by TMA, to rows that start anywhere."""
    _check(m, n, k, bias=True, act=act, residual=True, pre=True, layout=layout)
    _check(m, n, k, bias=True, act=act, residual=True, layout=layout, seed=62)
    wide = n // 2 if act == "geglu" else n
    _check(m, n, k, act=act, pre=True, layout=layout, out_ld=wide + 5, start=3, seed=63)


@pytest.mark.parametrize("n", [1024, 1022])
def test_long_sums_to_bf16_in_slices(n):
    _check(1024, n, 169151, layout=BOTH, bias=True, act="gelu", residual=True, pre=True)
