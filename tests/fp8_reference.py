"""Plain 64-bit forms of the 8-bit layer operators and the error bounds that
their tests use. Every bound is counted in roundings: a fp32 operation is off by
at most 2^-24 of its value, an output rounding by eps / 2 of its type."""

import torch

FLOOR = {torch.float8_e4m3fn: 2.0 ** -117, torch.float8_e5m2: 2.0 ** -110}
LARGEST = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
MANTISSA = {torch.float8_e4m3fn: 3, torch.float8_e5m2: 2}
LOWEST_EXPONENT = {torch.float8_e4m3fn: -6, torch.float8_e5m2: -14}
U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def scales_of(v, dtype, block_rows):
    """Scales [blocks of columns, blocks of rows] of a 64-bit matrix."""
    r, c = v.shape
    rb, cb = -(-r // block_rows), -(-c // 128)
    p = torch.zeros(rb * block_rows, cb * 128, dtype=torch.float64, device=v.device)
    p[:r, :c] = v.abs()
    amax = p.view(rb, block_rows, cb, 128).amax(dim=(1, 3))
    return (amax.clamp(min=FLOOR[dtype]) / LARGEST[dtype]).t()


def spread(scales, shape, block_rows):
    """One scale for every element of a matrix."""
    full = scales.t().repeat_interleave(block_rows, 0).repeat_interleave(128, 1)
    return full[:shape[0], :shape[1]]


def check_quantized(q, scales, v, dtype, block_rows, rel, what):
    """q and scales quantise the 64-bit matrix v when v itself is only known to
    `rel` of its value: the scale within rel plus its two roundings, and each
    element within half a step of the 8-bit grid plus rel, once through the block's
    maximum, and the four roundings of factor (three) and product."""
    want = scales_of(v, dtype, block_rows)
    assert scales.dtype == torch.float32 and scales.shape == want.shape, what
    assert q.dtype == dtype and q.shape == v.shape, what
    err = (scales.double() - want).abs()
    assert bool((err <= want * (rel + 2 * U)).all()), f"{what}: scales"
    target = v / spread(want, v.shape, block_rows)
    _, e = torch.frexp(target)
    step = torch.ldexp(torch.ones_like(target),
                       (e - 1).clamp(min=LOWEST_EXPONENT[dtype]) - MANTISSA[dtype])
    off = (q.double() - target).abs()
    worst = (off - step / 2 - (2 * rel + 4 * U) * target.abs()).max()
    assert float(worst) <= 0, f"{what}: {float(worst):.3e} beyond half a step"


def norm_depth(c):
    """Additions behind a row's sum, at most: 32 threads share a row, then the
    tree over a warp and the warps' sums in turn."""
    return c / 32 + 40


def rmsnorm(x, weight, eps, residual=None):
    """(y, h) in 64 bits; h is the sum as stored, in x's dtype."""
    h = x if residual is None else (x.double() + residual.double()).to(x.dtype)
    v = h.double()
    return v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps) * weight.double(), h


def rmsnorm_rel(c):
    """Relative error of y before its last rounding: half that of the sum of
    squares, then the division, the addition, the reciprocal root (two ulps) and
    two products."""
    return (norm_depth(c) / 2 + 10) * U


def rmsnorm_bwd(dy, h, weight, eps, dresidual=None):
    """(dx, dweight) in 64 bits and the magnitudes their errors scale with."""
    v, d, w = h.double(), dy.double(), weight.double()
    rstd = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps)
    n, g = v * rstd, d * w
    dx = rstd * (g - n * (g * n).mean(dim=1, keepdim=True))
    size = rstd * (g.abs() + n.abs() * (g * n).abs().mean(dim=1, keepdim=True))
    if dresidual is not None:
        dx = dx + dresidual.double()
        size = size + dresidual.double().abs()
    return dx, (d * n).sum(dim=0), size, (d * n).abs().sum(dim=0)


def matmul(a, a_scales, b, b_scales):
    """The product in 64 bits, and the same of magnitudes."""
    av = a.double() * spread(a_scales.double(), a.shape, 1)
    bv = b.double() * spread(b_scales.double(), b.shape, 128)
    return av @ bv.t(), av.abs() @ bv.abs().t()


def matmul_rel(k):
    """Error of the fp32 product relative to the product of magnitudes: 128
    products of a block are exact and are added in some order, each addition off
    by at most 2^-23 (rounded or cut off); then the product of scales, the
    scaling and the addition of each block."""
    return (128 * 2 + -(-k // 128) + 3) * U
