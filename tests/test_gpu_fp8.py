"""The 8-bit layer operators on the GPU against their definitions in 64 bits:
RMSNorm with residual and 8-bit output, its backward, quantisation, and the
block-scaled matrix product."""

import math

import pytest
import torch

import fp8_reference as ref
import padding_free_packed_gb300 as pe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
BF16, FP32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _fenced(rows, cols, dtype, fill, ld=None):
    """A matrix inside a buffer filled with `fill` (a byte): the caller checks
    that nothing outside the matrix changed."""
    size = torch.empty(0, dtype=dtype).element_size()
    ld = cols if ld is None else ld
    pad = 256                                   # keeps 16-byte alignment
    store = torch.full(((rows * ld * size + 2 * pad),), fill, dtype=torch.uint8, device=DEV)
    view = store[pad:pad + rows * ld * size].view(dtype).view(rows, ld)[:, :cols]
    return store, view


def _outside_untouched(store, rows, cols, dtype, fill, ld=None):
    size = torch.empty(0, dtype=dtype).element_size()
    ld = cols if ld is None else ld
    outside = store.clone()
    outside[256:256 + rows * ld * size].view(rows, ld * size)[:, :cols * size] = fill
    assert bool((outside == fill).all()), "bytes outside the matrix changed"


def _close(got, want, rel, dtype, what, size=None):
    """|got - want| <= rel * size (by default the value) + the output rounding."""
    got, want = got.double(), want.double()
    size = want.abs() if size is None else size
    bound = rel * size + (ref.half_step(dtype) if dtype != FP32 else ref.U) * want.abs() * (
        1 + 2 ** -8) + 1e-38
    worst = float(((got - want).abs() - bound).max()) if got.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} beyond the bound"


# ---------------------------------------------------------------- RMSNorm

WIDTHS = [1, 2, 7, 8, 63, 64, 127, 128, 129, 132, 255, 256, 257, 333, 500, 512, 768, 1000, 1024,
          1140, 1152, 1536, 2304, 2305, 4096, 9001]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("c", WIDTHS)
@pytest.mark.parametrize("with_residual", [False, True])
def test_rmsnorm(dtype, c, with_residual):
    gen = _gen(301)
    n = 37 if c > 600 else 301
    x = (_randn(gen, n, c) * 2).to(dtype)
    r = _randn(gen, n, c).to(dtype) if with_residual else None
    w = (1 + 0.3 * _randn(gen, c)).to(dtype)
    want, h = ref.rmsnorm(x, w, 1e-5, r)
    got = pe.pe_rmsnorm(x, w, 1e-5, residual=r)
    if with_residual:
        got, got_h = got
        assert torch.equal(got_h, h)
    _close(got, want, ref.rmsnorm_rel(c), dtype, f"rmsnorm c={c}")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("fp8", [E4M3, E5M2])
@pytest.mark.parametrize("c", WIDTHS)
def test_rmsnorm_fp8(dtype, fp8, c):
    gen = _gen(302)
    n = 41 if c > 600 else 300
    x = (_randn(gen, n, c) * torch.exp(_randn(gen, c))).to(dtype)
    r = _randn(gen, n, c).to(dtype)
    w = (1 + 0.3 * _randn(gen, c)).to(dtype)
    want, h = ref.rmsnorm(x, w, 1e-6, r)
    ld = (c + 15) // 16 * 16 + 16
    store, q = _fenced(n, c, fp8, 0x5A, ld)
    y = torch.empty_like(x)
    got, scales, got_h = pe.pe_rmsnorm_fp8(x, w, 1e-6, residual=r, dtype=fp8, out=q, y=y)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got_h, h)
    _outside_untouched(store, n, c, fp8, 0x5A, ld)
    ref.check_quantized(got, scales, want, fp8, 1, ref.rmsnorm_rel(c), f"rmsnorm_fp8 c={c}")
    _close(y, want, ref.rmsnorm_rel(c), dtype, f"y c={c}")
    plain, plain_scales = pe.pe_rmsnorm_fp8(h, w, 1e-6, dtype=fp8)     # the same without a residual
    assert torch.equal(plain.float(), got.float()) and torch.equal(plain_scales, scales)


# One width at least for every number of neighbouring channels an access can have (8, 4, 2,
# 1) and every number of warps a row is given; rows enough that a warp has several of them.
MANY = [(20011, 250), (20011, 255), (20011, 506), (20011, 501), (9001, 764), (9001, 758),
        (9001, 777), (5003, 1012), (5003, 1018), (5003, 1001), (5003, 1500), (5003, 1502),
        (5003, 1501), (2503, 1536), (2503, 2048), (5003, 2001), (2503, 2304), (2503, 2300),
        (2503, 2302), (2503, 2301), (2503, 2900), (2503, 2902), (2503, 2904), (2503, 4100)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,c", MANY)
def test_rmsnorm_of_many_rows(n, c, dtype):
    gen = _gen(308)
    x, r = (_randn(gen, n, c) * 2).to(dtype), _randn(gen, n, c).to(dtype)
    w = (1 + 0.3 * _randn(gen, c)).to(dtype)
    want, h = ref.rmsnorm(x, w, 1e-5, r)
    y = torch.empty_like(x)
    q, scales, got_h = pe.pe_rmsnorm_fp8(x, w, 1e-5, residual=r, y=y)
    assert torch.equal(got_h, h)
    _close(y, want, ref.rmsnorm_rel(c), dtype, f"y {n} x {c}")
    ref.check_quantized(q, scales, want, E4M3, 1, ref.rmsnorm_rel(c), f"rmsnorm_fp8 {n} x {c}")
    few = pe.pe_rmsnorm_fp8(x[:3], w, 1e-5, residual=r[:3])       # a row's bits are its own
    assert torch.equal(few[0].float(), q[:3].float()) and torch.equal(few[1], scales[:, :3])
    plain, got_h = pe.pe_rmsnorm(x, w, 1e-5, residual=r, out=x, residual_out=r)   # in place
    assert torch.equal(plain, y) and torch.equal(r, h) and got_h.data_ptr() == r.data_ptr()


@pytest.mark.parametrize("c", [768, 1001, 9000])
def test_rmsnorm_in_place(c):
    """residual_out may be the residual's buffer and y may be x's."""
    gen = _gen(303)
    x, r = _randn(gen, 70, c).to(BF16), _randn(gen, 70, c).to(BF16)
    w = (1 + 0.3 * _randn(gen, c)).to(BF16)
    y, h = pe.pe_rmsnorm(x, w, residual=r)
    q, s, _ = pe.pe_rmsnorm_fp8(x, w, residual=r)
    x2, r2 = x.clone(), r.clone()
    got, got_h = pe.pe_rmsnorm(x2, w, residual=r2, out=x2, residual_out=r2)
    assert got.data_ptr() == x2.data_ptr() and got_h.data_ptr() == r2.data_ptr()
    assert torch.equal(x2, y) and torch.equal(r2, h)
    x3, r3 = x.clone(), r.clone()
    q3, s3, _ = pe.pe_rmsnorm_fp8(x3, w, residual=r3, y=r3, residual_out=x3)
    assert torch.equal(x3, h) and torch.equal(r3, y)
    assert torch.equal(q3.float(), q.float()) and torch.equal(s3, s)


def test_rmsnorm_of_rows_with_nothing_in_them():
    """Zero rows give zeros and the smallest scale; NaN and infinities stay in
    their own rows."""
    gen = _gen(304)
    x = _randn(gen, 6, 300).to(BF16)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 290] = float("inf")
    w = torch.ones(300, dtype=BF16, device=DEV)
    q, s = pe.pe_rmsnorm_fp8(x, w)
    assert bool((q[1].float() == 0).all())
    assert bool((s[:, 1] == torch.tensor(ref.FLOOR[E4M3] / 448, device=DEV).float()).all())
    assert bool(q[2].float().isnan().all()) and bool(s[:, 2].isnan().all())
    assert bool(q[3, 290].float().isnan()) and bool(s[2, 3].isnan())
    clean = x[[0, 4, 5]].contiguous()
    qc, sc = pe.pe_rmsnorm_fp8(clean, w)
    assert torch.equal(q[[0, 4, 5]].float(), qc.float()) and torch.equal(s[:, [0, 4, 5]], sc)


@pytest.mark.parametrize("c", [768, 333])
def test_rmsnorm_sums_of_the_smallest_and_largest_numbers(c):
    """The stored sum is the fp32 sum rounded to bf16 also for subnormal numbers,
    sums that cancel, overflow, and infinities."""
    x = _randn(_gen(307), 64, c).to(BF16)
    r = _randn(_gen(308), 64, c).to(BF16)
    x[:8] *= 2.0 ** -132
    r[:8] *= 2.0 ** -133
    x[8:16] = -r[8:16]
    x[16:24] *= 2.0 ** -20
    x[24:32], r[24:32] = 3e38, 3e38
    x[32:40, ::3] = float("inf")
    r[36:40, ::3] = float("-inf")
    w = torch.ones(c, dtype=BF16, device=DEV)
    want = (x.float() + r.float()).to(BF16)
    _, h = pe.pe_rmsnorm(x, w, residual=r)
    _, _, h8 = pe.pe_rmsnorm_fp8(x, w, residual=r)
    for got in (h, h8):
        assert torch.equal(got.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


def test_rmsnorm_without_rows():
    x = torch.empty(0, 64, dtype=BF16, device=DEV)
    w = torch.ones(64, dtype=BF16, device=DEV)
    assert pe.pe_rmsnorm(x, w).shape == (0, 64)
    q, s = pe.pe_rmsnorm_fp8(x, w)
    assert q.shape == (0, 64) and s.shape == (1, 0)
    dx, dw = pe.pe_rmsnorm_bwd(x, x, w)
    assert dx.shape == (0, 64) and bool((dw == 0).all())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("c", [1, 3, 64, 127, 256, 333, 512, 768, 1000, 1001, 1024, 2304, 2500, 4096,
                               5000, 5001, 16384])
@pytest.mark.parametrize("n,with_residual", [(1, True), (1777, False), (700, True)])
def test_rmsnorm_bwd(dtype, c, n, with_residual):
    gen = _gen(305)
    h = (_randn(gen, n, c) * 1.5).to(dtype)
    dy = _randn(gen, n, c).to(dtype)
    w = (1 + 0.3 * _randn(gen, c)).to(dtype)
    dr = _randn(gen, n, c).to(dtype) if with_residual else None
    dx, dw = pe.pe_rmsnorm_bwd(dy, h, w, 1e-5, dresidual=dr)
    want_dx, want_dw, size, dw_size = ref.rmsnorm_bwd(dy, h, w, 1e-5, dr)
    # rstd enters dx up to three times, with half the error of its sum.
    _close(dx, want_dx, (2.5 * ref.norm_depth(c) + 24) * ref.U, dtype, "dx", size)
    # A thread adds the rows of one of at least 152 blocks, then warps and blocks.
    rel = (n / 152 + 1 + 24 + ref.norm_depth(c) / 2 + 10) * ref.U
    assert dw.dtype == FP32
    _close(dw, want_dw, rel, FP32, "dweight", dw_size)
    again, dw_again = pe.pe_rmsnorm_bwd(dy, h, w, 1e-5, dresidual=dr)
    assert torch.equal(dx, again) and torch.equal(dw, dw_again)
    into = dy.clone()                                           # dx over dy
    over, _ = pe.pe_rmsnorm_bwd(into, h, w, 1e-5, dresidual=dr, out=into)
    assert torch.equal(over, dx)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,c", MANY)
def test_rmsnorm_bwd_of_many_rows(n, c, dtype):
    gen = _gen(309)
    h, dy = (_randn(gen, n, c) * 1.5).to(dtype), _randn(gen, n, c).to(dtype)
    w = (1 + 0.3 * _randn(gen, c)).to(dtype)
    dr = _randn(gen, n, c).to(dtype)
    want_dx, want_dw, size, dw_size = ref.rmsnorm_bwd(dy, h, w, 1e-5, dr)
    dx, dw = pe.pe_rmsnorm_bwd(dy, h, w, 1e-5, dresidual=dr)
    _close(dx, want_dx, (2.5 * ref.norm_depth(c) + 24) * ref.U, dtype, "dx", size)
    rel = (n / 152 + 1 + 24 + ref.norm_depth(c) / 2 + 10) * ref.U     # as above
    _close(dw, want_dw, rel, FP32, "dweight", dw_size)
    few, _ = pe.pe_rmsnorm_bwd(dy[:3], h[:3], w, 1e-5, dresidual=dr[:3])
    assert torch.equal(few, dx[:3])
    over, dw_over = pe.pe_rmsnorm_bwd(dy, h, w, 1e-5, dresidual=dr, out=dy)       # dx over dy
    assert torch.equal(over, dx) and torch.equal(dw_over, dw)


def test_rmsnorm_bwd_against_differences():
    """Central differences of a scalar of the fp32 forward. Step e = 2^-6 on one
    input: the difference quotient is off by e^2/6 |f'''| plus the forward's
    rounding, 2 * rel * sum|g y| / (2 e); third derivatives of y in one channel
    are at most 15 |g|_1 (max|h| / rms + 1)^3 rstd^3."""
    gen = _gen(306)
    n, c, e = 5, 48, 2.0 ** -6
    h, g = _randn(gen, n, c), _randn(gen, n, c)
    w = 1 + 0.3 * _randn(gen, c)
    dx, dw = pe.pe_rmsnorm_bwd(g, h, w, 1e-3)

    def f(hh, ww):
        y = pe.pe_rmsnorm(hh, ww, 1e-3)
        return float((y.double() * g.double()).sum())

    rstd = 1 / math.sqrt(float((h.double() ** 2).mean(dim=1).min()))
    big = float(h.abs().max())
    noise = ref.rmsnorm_rel(c) * float((pe.pe_rmsnorm(h, w, 1e-3) * g).abs().sum()) / e
    third = e * e / 6 * 15 * float(g.abs().sum(dim=1).max()) * 2 * (big * rstd + 1) ** 3 * rstd ** 3
    for row, col in [(0, 0), (2, 17), (4, 47)]:
        up, down = h.clone(), h.clone()
        up[row, col] += e
        down[row, col] -= e
        width = float(up[row, col].double() - down[row, col].double())
        slope = (f(up, w) - f(down, w)) / width
        assert abs(slope - float(dx[row, col])) <= noise + third + 1e-5
        up, down = w.clone(), w.clone()
        up[col] += e
        down[col] -= e
        width = float(up[col].double() - down[col].double())
        slope = (f(h, up) - f(h, down)) / width                  # linear in the weight
        assert abs(slope - float(dw[col])) <= noise + 1e-5


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("fp8", [E4M3, E5M2])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 768), (3, 129), (16, 128), (127, 64), (128, 128),
                                       (130, 260), (257, 1001), (768, 500), (301, 2304), (1000, 7)])
def test_quantize(dtype, fp8, block_rows, rows, cols):
    gen = _gen(311)
    x = (_randn(gen, rows, cols) * torch.exp(2 * _randn(gen, cols))).to(dtype)
    q, s, qt, st = pe.pe_quantize_fp8(x, block_rows, dtype=fp8, plain=True, transposed=True)
    ref.check_quantized(q, s, x.double(), fp8, block_rows, 0.0, "as it is")
    ref.check_quantized(qt, st, x.double().t(), fp8, block_rows, 0.0, "transposed")
    if block_rows == 128:
        assert torch.equal(qt.float(), q.float().t()) and torch.equal(st, s.t())
    only = pe.pe_quantize_fp8(x, block_rows, dtype=fp8)
    only_t = pe.pe_quantize_fp8(x, block_rows, dtype=fp8, plain=False, transposed=True)
    for got, want in zip(only + only_t, (q, s, qt, st)):
        assert torch.equal(got.float(), want.float())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 130), (129, 3), (140, 256), (257, 253), (300, 390),
                                       (384, 131)])
def test_quantize_of_rows_that_start_anywhere(rows, cols, offset, block_rows, dtype):
    """A matrix at any element of a buffer; what lies around it is not used."""
    buffer = torch.full((rows * cols + 16,), float("nan"), device=DEV, dtype=dtype)
    x = buffer[offset:offset + rows * cols].view(rows, cols)
    x.copy_(_randn(_gen(315), rows, cols) * torch.exp(2 * _randn(_gen(316), cols)))
    q, s, qt, st = pe.pe_quantize_fp8(x, block_rows, transposed=True)
    ref.check_quantized(q, s, x.double(), E4M3, block_rows, 0.0, "as it is")
    ref.check_quantized(qt, st, x.double().t(), E4M3, block_rows, 0.0, "transposed")


@pytest.mark.parametrize("rows,cols", [(37, 100), (128, 33), (200, 384)])
def test_quantize_writes_nothing_outside(rows, cols):
    """The C entry with leading dimensions of its own and guarded buffers."""
    x = _randn(_gen(312), rows, cols)
    lib = pe.load_library()
    ld, ldt = (cols + 15) // 16 * 16 + 32, (rows + 15) // 16 * 16 + 16
    store, q = _fenced(rows, cols, E4M3, 0x33, ld)
    store_t, qt = _fenced(cols, rows, E4M3, 0x33, ldt)
    cb, rb = -(-cols // 128), -(-rows // 128)
    ss, s = _fenced(cb, rows, FP32, 0x33)
    sst, st = _fenced(rb, cols, FP32, 0x33)
    assert lib.pe_quantize_fp8(1, 0, x.data_ptr(), rows, cols, 1, q.data_ptr(), ld, s.data_ptr(),
                               qt.data_ptr(), ldt, st.data_ptr(),
                               torch.cuda.current_stream().cuda_stream) == 0
    ref.check_quantized(q, s, x.double(), E4M3, 1, 0.0, "as it is")
    ref.check_quantized(qt, st, x.double().t(), E4M3, 1, 0.0, "transposed")
    _outside_untouched(store, rows, cols, E4M3, 0x33, ld)
    _outside_untouched(store_t, cols, rows, E4M3, 0x33, ldt)
    _outside_untouched(ss, cb, rows, FP32, 0x33)
    _outside_untouched(sst, rb, cols, FP32, 0x33)


@pytest.mark.parametrize("fp8", [E4M3, E5M2])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_of_the_smallest_and_largest_blocks(block_rows, dtype, fp8):
    """Blocks of zeros, of the smallest and of the largest numbers of the type."""
    x = _randn(_gen(314), 384, 128).clamp(-3, 3).to(dtype)
    x[:128] = 0
    x[128:256] *= 2.0 ** -116                   # around both floors
    x[256:] *= 2.0 ** 126
    for v in (x, x.t().contiguous()):
        q, s, qt, st = pe.pe_quantize_fp8(v, block_rows, dtype=fp8, transposed=True)
        ref.check_quantized(q, s, v.double(), fp8, block_rows, 0.0, "as it is")
        ref.check_quantized(qt, st, v.double().t(), fp8, block_rows, 0.0, "transposed")
    q, s = pe.pe_quantize_fp8(x, block_rows, dtype=fp8)
    assert bool((q[:128].float() == 0).all())
    w = torch.ones(128, dtype=dtype, device=DEV)
    zero, zs = pe.pe_rmsnorm_fp8(torch.zeros_like(x), w, dtype=fp8)
    assert bool((zero.float() == 0).all()) and bool(zs.isfinite().all())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_of_special_values(block_rows):
    x = _randn(_gen(313), 256, 256)
    x[:128, :128] = 0
    x[128:, :128] *= 1e-38                      # far below the smallest block magnitude
    x[0, 200] = float("nan")
    x[200, 250] = float("-inf")
    q, s = pe.pe_quantize_fp8(x, block_rows)
    per = ref.spread(s.double(), x.shape, block_rows)
    back = q.double() * per
    assert bool((q[:128, :128].float() == 0).all())
    # 1e-38 |N(0,1)| times 448 / 2^-117 = 7.4e37 is of the order of 1: small
    # numbers of the grid, not zeros.
    ref.check_quantized(q[:, :128], s[:1], x[:, :128].double(), E4M3, block_rows, 0.0, "tiny")
    assert bool((s[0] == torch.tensor(ref.FLOOR[E4M3] / 448, device=DEV).float()).all())
    if block_rows == 128:
        assert bool(back[:, 128:].isnan().all())
    else:
        assert bool(back[0, 128:].isnan().all()) and bool(back[200, 128:].isnan().all())
        rest = [i for i in range(256) if i not in (0, 200)]
        assert bool(back[rest].isfinite().all())


# ---------------------------------------------------------------- matrix product

SHAPES = [(1, 1, 1), (1, 2304, 768), (1, 64, 16), (2, 129, 100), (7, 1152, 768), (8, 8, 128),
          (16, 128, 127), (17, 300, 129), (31, 1001, 640), (33, 64, 2304), (64, 768, 1152),
          (65, 96, 4101), (100, 2304, 768), (127, 127, 127), (128, 128, 128), (129, 257, 255),
          (200, 768, 768), (255, 500, 1024), (256, 256, 256), (257, 1000, 300), (320, 1001, 1140),
          (512, 512, 512), (640, 2304, 768), (1000, 999, 1001), (1537, 768, 1152),
          (3000, 2304, 768), (5001, 100, 64), (4999, 1024, 1024), (768, 768, 9001),
          (2304, 768, 4097), (64, 64, 32299), (1, 1, 32299), (300, 130, 20000),
          (9000, 64, 100), (20000, 512, 512), (40001, 256, 72), (1, 33000, 96)]


def _operands(gen, m, n, k, ta=E4M3, tb=E4M3, ints=False):
    """Quantised operands in buffers whose padding bytes and surrounding rows
    hold NaN codes."""
    lda, ldb = (k + 15) // 16 * 16 + 16, (k + 15) // 16 * 16
    _, a = _fenced(m, k, ta, 0x7F, lda)
    _, b = _fenced(n, k, tb, 0x7F, ldb)
    kb, nb = -(-k // 128), -(-n // 128)
    if ints:
        a.copy_(torch.randint(-1, 2, (m, k), generator=gen, device=DEV).float())
        b.copy_(torch.randint(-1, 2, (n, k), generator=gen, device=DEV).float())
        sa = torch.exp2(torch.randint(-1, 2, (kb, m), generator=gen, device=DEV).float())
        sb = torch.exp2(torch.randint(-1, 2, (kb, nb), generator=gen, device=DEV).float())
        return a, sa, b, sb
    qa, sa = pe.pe_quantize_fp8(_randn(gen, m, k) * torch.exp(_randn(gen, k)), 1, dtype=ta)
    qb, sb = pe.pe_quantize_fp8(_randn(gen, n, k), 128, dtype=tb)
    a.copy_(qa)
    b.copy_(qb)
    return a, sa, b, sb


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul_of_small_whole_numbers_is_exact(m, n, k):
    """Operands -1, 0, 1 and scales 1/2, 1, 2: every partial sum is a multiple
    of 1/4 below 2^20, so fp32 holds it and the product has no rounding at all.
    The fp32 output, its guard bytes and the bf16 output are checked."""
    a, sa, b, sb = _operands(_gen(321), m, n, k, ints=True)
    want, _ = ref.matmul(a, sa, b, sb)
    store, out = _fenced(m, n, FP32, 0x77)
    pe.pe_matmul_fp8(a, sa, b, sb, out=out)
    assert torch.equal(out.double(), want)
    _outside_untouched(store, m, n, FP32, 0x77)
    store, out = _fenced(m, n, BF16, 0x77)
    pe.pe_matmul_fp8(a, sa, b, sb, out=out)
    assert torch.equal(out, want.float().to(BF16))
    _outside_untouched(store, m, n, BF16, 0x77)
    assert pe.pe_read_matmul_status() == 0


@pytest.mark.parametrize("ta,tb", [(E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2)])
@pytest.mark.parametrize("m,n,k", [(1, 300, 768), (40, 1001, 500), (320, 1001, 1140),
                                   (1111, 768, 1152), (4000, 2304, 768), (768, 640, 9001)])
def test_matmul(ta, tb, m, n, k):
    a, sa, b, sb = _operands(_gen(322), m, n, k, ta, tb)
    want, size = ref.matmul(a, sa, b, sb)
    for dtype in (FP32, BF16):
        out = pe.pe_matmul_fp8(a, sa, b, sb, dtype=dtype)
        assert out.dtype == dtype
        _close(out, want, ref.matmul_rel(k), dtype, f"matmul {dtype}", size)
        assert torch.equal(out, pe.pe_matmul_fp8(a, sa, b, sb, dtype=dtype))


def test_matmul_with_nothing_to_sum_or_to_write():
    empty = torch.empty(5, 0, dtype=E4M3, device=DEV)
    w = torch.empty(3, 0, dtype=E4M3, device=DEV)
    out = pe.pe_matmul_fp8(empty, torch.empty(0, 5, device=DEV), w, torch.empty(0, 1, device=DEV))
    assert out.shape == (5, 3) and bool((out == 0).all())
    a, sa, b, sb = _operands(_gen(323), 4, 64, 128)
    none = torch.empty(0, 128, dtype=E4M3, device=DEV)
    assert pe.pe_matmul_fp8(none, torch.empty(1, 0, device=DEV), b, sb).shape == (0, 64)
    assert pe.pe_matmul_fp8(a, sa, none, torch.empty(1, 0, device=DEV)).shape == (4, 0)


@pytest.mark.parametrize("m", [3, 300, 3000])
def test_matmul_keeps_nan_in_its_rows_and_columns(m):
    a, sa, b, sb = _operands(_gen(324), m, 400, 300)
    want = pe.pe_matmul_fp8(a, sa, b, sb)
    a, sa = a.clone(), sa.clone()
    a.view(torch.uint8)[1, 17] = 0x7F
    sa[2, 0] = float("inf")
    got = pe.pe_matmul_fp8(a, sa, b, sb)
    assert bool(got[1].isnan().all()) and not bool(got[0].isfinite().any())
    assert torch.equal(got[2:], want[2:])


def test_matmul_takes_operands_of_any_layout():
    """Operands whose rows do not start at 16-byte multiples are laid out first."""
    gen = _gen(325)
    a, sa, b, sb = _operands(gen, 50, 70, 100)
    want = pe.pe_matmul_fp8(a, sa, b, sb)
    tight = a.contiguous()
    assert tight.stride(0) == 100
    assert torch.equal(pe.pe_matmul_fp8(tight, sa, b, sb), want)
    assert torch.equal(pe.pe_matmul_fp8(a, sa, b.t().contiguous().t(), sb), want)
    assert torch.equal(pe.pe_matmul_fp8(a, sa.t().contiguous().t(), b, sb), want)


@pytest.mark.parametrize("m,n,k", [(5, 2304, 768), (700, 768, 768), (3000, 1024, 1024),
                                   (768, 768, 9001)])
def test_matmul_on_two_streams_at_once(m, n, k):
    sets = [_operands(_gen(326 + i), m, n, k) for i in range(2)]
    want = [pe.pe_matmul_fp8(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(pe.pe_matmul_fp8(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert torch.equal(out, want[i])
    assert pe.pe_read_matmul_status() == 0


# ---------------------------------------------------------------- together

def _layer(x, residual, w, eps):
    """Norm, up projection, GeGLU, down projection, all linear steps in 8 bits."""
    q, s, h = pe.pe_rmsnorm_fp8(x, w["norm"], eps, residual=residual)
    up = pe.pe_matmul_fp8(q, s, *w["up"])
    act, act_s = pe.pe_quantize_fp8(pe.pe_geglu(up))
    return pe.pe_matmul_fp8(act, act_s, *w["down"]), h


def _weights(gen, c, f):
    up, down = _randn(gen, 2 * f, c) / math.sqrt(c), _randn(gen, c, f) / math.sqrt(f)
    return {"norm": (1 + 0.2 * _randn(gen, c)).to(BF16),
            "up": pe.pe_quantize_fp8(up.to(BF16), 128),
            "down": pe.pe_quantize_fp8(down.to(BF16), 128)}


@pytest.mark.parametrize("n", [1, 320, 5000])
def test_layer_steps_follow_each_other(n):
    """Each step of the chain against its 64-bit form on the same inputs."""
    gen = _gen(331)
    c, f = 768, 1152
    w = _weights(gen, c, f)
    x, r = _randn(gen, n, c).to(BF16), _randn(gen, n, c).to(BF16)
    y, h = ref.rmsnorm(x, w["norm"], 1e-5, r)
    q, s, got_h = pe.pe_rmsnorm_fp8(x, w["norm"], 1e-5, residual=r)
    assert torch.equal(got_h, h)
    ref.check_quantized(q, s, y, E4M3, 1, ref.rmsnorm_rel(c), "norm")
    up = pe.pe_matmul_fp8(q, s, *w["up"])
    want, size = ref.matmul(q, s, *w["up"])
    _close(up, want, ref.matmul_rel(c), BF16, "up", size)
    act = pe.pe_geglu(up)
    act_q, act_s = pe.pe_quantize_fp8(act)
    ref.check_quantized(act_q, act_s, act.double(), E4M3, 1, 0.0, "activation")
    out = pe.pe_matmul_fp8(act_q, act_s, *w["down"])
    want, size = ref.matmul(act_q, act_s, *w["down"])
    _close(out, want, ref.matmul_rel(f), BF16, "down", size)
    chained, chained_h = _layer(x, r, w, 1e-5)
    assert torch.equal(chained, out) and torch.equal(chained_h, h)


@pytest.mark.parametrize("n", [3, 900, 5000])
def test_layer_in_a_cuda_graph(n):
    gen = _gen(332)
    w = _weights(gen, 512, 640)
    x, r = _randn(gen, n, 512).to(BF16), _randn(gen, n, 512).to(BF16)
    _layer(x, r, w, 1e-5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, h = _layer(x, r, w, 1e-5)
    for _ in range(3):
        x.copy_(_randn(gen, n, 512))
        r.copy_(_randn(gen, n, 512))
        graph.replay()
        want, want_h = _layer(x.clone(), r.clone(), w, 1e-5)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(h, want_h)


def test_training_step_of_a_linear_layer():
    """Y = norm(X) W^T and its gradients from quantised operands: every product
    against the 64-bit product of the same operands, and the whole within what
    8-bit rounding of both operands allows: each element off by at most its half
    step, 2^-4 relative for e4m3 and 2^-3 for e5m2, plus the grid's lower end."""
    gen = _gen(333)
    n, c, m = 1300, 512, 384
    x = _randn(gen, n, c).to(BF16)
    wn = (1 + 0.2 * _randn(gen, c)).to(BF16)
    wt = (_randn(gen, m, c) / math.sqrt(c)).to(BF16)
    dy = _randn(gen, n, m).to(BF16)
    y = torch.empty_like(x)
    q, s = pe.pe_rmsnorm_fp8(x, wn, y=y)
    wq, ws, wtq, wts = pe.pe_quantize_fp8(wt, 128, transposed=True)
    out = pe.pe_matmul_fp8(q, s, wq, ws)
    gq, gs, gtq, gts = pe.pe_quantize_fp8(dy, 1, dtype=E5M2, transposed=True)
    ytq, yts = pe.pe_quantize_fp8(y, 128, plain=False, transposed=True)
    d_norm = pe.pe_matmul_fp8(gq, gs, wtq, wts)
    d_w = pe.pe_matmul_fp8(gtq, gts, ytq, yts, dtype=FP32)
    dx, d_wn = pe.pe_rmsnorm_bwd(d_norm, x, wn)
    for got, ops, depth in ((out, (q, s, wq, ws), c), (d_norm, (gq, gs, wtq, wts), m),
                            (d_w, (gtq, gts, ytq, yts), n)):
        want, size = ref.matmul(*ops)
        _close(got, want, ref.matmul_rel(depth), got.dtype, "product", size)
    want_dx, want_dwn, size, dw_size = ref.rmsnorm_bwd(d_norm, x, wn, 1e-5)
    _close(dx, want_dx, (2.5 * ref.norm_depth(c) + 24) * ref.U, BF16, "dx", size)
    # Against the unquantised product: an operand's block maximum is at most the
    # largest value there is, so its grid ends at 2^-10 (e4m3) or 2^-17 (e5m2) of F.
    yn = y.double()
    full, full_size = dy.double().t() @ yn, dy.double().abs().t() @ yn.abs()
    rel_g, rel_y = 2.0 ** -3, 2.0 ** -4
    floor_g = float(dy.abs().max()) / 57344 * 2.0 ** -17
    floor_y = float(y.abs().max()) / 448 * 2.0 ** -10
    bound = ((1 + rel_g) * (1 + rel_y) - 1) * full_size + 1.2 * (
        floor_g * yn.abs().sum(dim=0)[None, :] + floor_y * dy.double().abs().sum(dim=0)[:, None])
    bound = bound + 1.2 * n * floor_g * floor_y + 2.0 ** -8 * full_size
    assert bool(((d_w.double() - full).abs() <= bound).all())
