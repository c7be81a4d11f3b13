"""Quantisation against IEEE division: a block's scale is amax / F and its factor
F / amax, each the fp32 number nearest to the quotient, so that scales and values
equal bit for bit what the same fp32 operations give on the host (the factor and
the product with it, one rounding each, then the rounding to 8 bits)."""

import pytest
import torch

import fp8_reference as ref
import padding_free_packed_gb300 as pe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
BF16, FP32 = torch.bfloat16, torch.float32


def _by_division(x, dtype, block_rows):
    """(values as fp32, scales) of x quantised on the host in fp32."""
    x = x.cpu().float()
    r, c = x.shape
    rb, cb = -(-r // block_rows), -(-c // 128)
    p = torch.zeros(rb * block_rows, cb * 128)
    p[:r, :c] = x
    p = p.view(rb, block_rows, cb, 128)
    amax = p.abs().amax(dim=(1, 3)).clamp(min=ref.FLOOR[dtype])
    # Tensor by tensor: a quotient with a Python number is a product with a reciprocal.
    largest = torch.full_like(amax, ref.LARGEST[dtype])
    q = p * torch.div(largest, amax)[:, None, :, None]
    return q.reshape(rb * block_rows, -1)[:r, :c].to(dtype).float(), torch.div(amax, largest).t()


def _rows(seed, rows, cols, spread):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    return x * torch.exp(spread * torch.randn(rows, 1, generator=gen, device=DEV))


@pytest.mark.parametrize("fp8", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(257, 1001), (2304, 768), (1500, 132)])
def test_quantize_divides_as_ieee_does(rows, cols, block_rows, dtype, fp8):
    x = _rows(501, rows, cols, 8).to(dtype)
    x[3] = 0
    q, s, qt, st = pe.pe_quantize_fp8(x, block_rows, dtype=fp8, transposed=True)
    for got, scales, v in ((q, s, x), (qt, st, x.t())):
        want, want_scales = _by_division(v, fp8, block_rows)
        assert torch.equal(scales.cpu(), want_scales)
        assert torch.equal(got.cpu().float(), want)


@pytest.mark.parametrize("fp8", [E4M3, E5M2])
@pytest.mark.parametrize("cols", [500, 768, 1001, 9001])
def test_the_norm_quantises_its_output_as_ieee_does(cols, fp8):
    """With fp32 rows y is the unrounded output that the 8-bit values come from."""
    x = _rows(502, 300, cols, 1)
    w = 1 + 0.3 * _rows(503, 1, cols, 0)[0]
    y = torch.empty_like(x)
    q, s = pe.pe_rmsnorm_fp8(x, w, dtype=fp8, y=y)
    want, want_scales = _by_division(y, fp8, 1)
    assert torch.equal(s.cpu(), want_scales)
    assert torch.equal(q.cpu().float(), want)
