"""The 8-bit product where the product of two scales leaves the range of fp32
although the result does not: blocks of the smallest and largest magnitudes that
quantisation makes, next to ordinary ones."""

import pytest
import torch

import fp8_reference as ref
import padding_free_packed_gb300 as pe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
BF16, FP32 = torch.bfloat16, torch.float32

# Every kernel form: 16, 32 and 64 rows a CTA, without and with a split sum; pairs on
# whole tiles with each form of output; pairs that share tiles, even and ragged.
WAYS = [(5, 300, 500), (3, 512, 4000), (320, 1001, 1140), (300, 130, 20000), (1537, 768, 1152),
        (768, 768, 4500), (768, 768, 9001), (9000, 1152, 768), (9000, 1001, 768),
        (2304, 768, 20000), (2500, 999, 9001)]


def _operands(m, n, k, low, high):
    """e5m2 operands with 4-bit numbers from 2^low to 2^high."""
    gen = torch.Generator(device=DEV).manual_seed(511)

    def values(rows, cols):
        e = torch.randint(low, high, (rows, cols), generator=gen, device=DEV).float()
        v = torch.exp2(e) * (1 + 0.25 * torch.randint(0, 4, (rows, cols), generator=gen, device=DEV))
        sign = torch.randint(0, 2, (rows, cols), generator=gen, device=DEV).float() * 2 - 1
        return (v * sign).to(E5M2)

    def scales(*shape):
        return 1 + torch.rand(*shape, generator=gen, device=DEV)

    kb = -(-k // 128)
    return values(m, k), scales(kb, m), values(n, k), scales(kb, -(-n // 128)), gen


def _check(a, sa, b, sb, dtype):
    k = a.shape[1]
    want, size = ref.matmul(a, sa, b, sb)
    got = pe.pe_matmul_fp8(a, sa, b, sb, dtype=dtype)
    assert pe.pe_read_matmul_status() == 0
    # Below 2^-126 a rounding is off by half of the last place there, 2^-150 (bf16: 2^-134):
    # one for each block's addition, one for the output.
    tiny = (-(-k // 128) + 1) * 2.0 ** -150 + (2.0 ** -134 if dtype == BF16 else 0)
    half = ref.half_step(dtype) if dtype == BF16 else 0
    rel = ref.matmul_rel(k) + 1 * ref.U                # one product of scales more
    bound = rel * size + half * (want.abs() + rel * size) + tiny
    assert bool(((got.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("m,n,k", WAYS)
@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_blocks_of_the_smallest_magnitudes(m, n, k, dtype):
    """A block at the floor of its scale (2^-126 or so) against a weight of ordinary
    size: the product of scales is below 2^-126, the result is not."""
    a, sa, b, sb, _ = _operands(m, n, k, 2, 12)
    _check(a, sa * 2.0 ** -126, b, sb * 2.0 ** -14, dtype)


@pytest.mark.parametrize("m,n,k", WAYS)
def test_blocks_of_the_largest_magnitudes(m, n, k):
    """The product of scales is above 2^128; results are near 2^120, or zero where a
    row holds zeros."""
    a, sa, b, sb, _ = _operands(m, n, k, -14, -9)
    a[::3] = 0
    _check(a, sa * 2.0 ** 100, b, sb * 2.0 ** 36, FP32)
    assert bool((pe.pe_matmul_fp8(a, sa * 2.0 ** 100, b, sb * 2.0 ** 36)[::3] == 0).all())


@pytest.mark.parametrize("m,n,k", WAYS)
def test_blocks_of_every_magnitude_side_by_side(m, n, k):
    a, sa, b, sb, gen = _operands(m, n, k, -14, -9)

    def mixed(s, exponents):
        pick = torch.randint(0, len(exponents), s.shape, generator=gen, device=DEV)
        return s * torch.exp2(torch.tensor(exponents, device=DEV, dtype=FP32))[pick]

    _check(a, mixed(sa, [-126.0, -30.0, 0.0, 100.0]), b, mixed(sb, [-14.0, 0.0, 36.0]), FP32)


@pytest.mark.parametrize("m,n,k", WAYS)
def test_a_row_does_not_depend_on_blocks_beside_it(m, n, k):
    """Ordinary rows next to rows of the smallest magnitudes keep their bits."""
    a, sa, b, sb, _ = _operands(m, n, k, -4, 4)
    want = pe.pe_matmul_fp8(a, sa, b, sb, dtype=FP32)
    far = sa.clone()
    far[:, 1::2] *= 2.0 ** -126
    small = sb * 2.0 ** -14
    got = pe.pe_matmul_fp8(a, far * 2.0 ** 0, b, small, dtype=FP32)
    assert torch.equal(got[::2] * 2.0 ** 14, want[::2])


@pytest.mark.parametrize("m,n,k", [(5, 300, 500), (9000, 1001, 768)])
def test_scales_that_are_not_numbers_and_zeros(m, n, k):
    """By the formula: an infinite or NaN scale spoils its row, a zero one its block only."""
    a, sa, b, sb, _ = _operands(m, n, k, -4, 4)
    want = pe.pe_matmul_fp8(a, sa, b, sb, dtype=FP32)
    sa[1, 0], sa[0, 1], sa[:, 2] = float("inf"), float("nan"), 0.0
    got = pe.pe_matmul_fp8(a, sa, b, sb, dtype=FP32)
    assert not bool(got[0].isfinite().any()) and bool(got[1].isnan().all())
    assert bool((got[2] == 0).all()) and torch.equal(got[3:], want[3:])


@pytest.mark.parametrize("m,n,k", WAYS)
def test_infinite_operands_next_to_far_scales(m, n, k):
    """e5m2 has infinities: a row that holds one is infinite as the formula says, whatever
    the scales of the rows beside it, and no number where its own block's are far."""
    a, sa, b, sb, _ = _operands(m, n, k, -4, 4)
    a, sa = a.clone(), sa.clone()
    a[0, 0], a[1, 0], a[2, k - 1] = float("inf"), float("-inf"), float("inf")
    sa[0, 1] *= 2.0 ** -126
    sa[-1, 2] *= 2.0 ** 126
    for small in (sb * 2.0 ** -14, sb * 2.0 ** 10):
        got = pe.pe_matmul_fp8(a, sa, b, small, dtype=FP32)
        want, _ = ref.matmul(a, sa, b, small)
        assert torch.equal(got[:1].double(), want[:1]) and bool(got[0].isinf().all())
        assert not bool(got[1:3].isfinite().any())
        assert bool(got[3:].isfinite().all())
