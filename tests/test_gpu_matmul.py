"""The 16- and 32-bit matrix product with its epilogue on the GPU against its definition in 64
bits."""

import pytest
import torch

import padding_free_packed_gb300 as pe
import tail_reference as ref
from tail_reference import U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
LAYOUTS = [(False, False), (False, True), (True, False), (True, True)]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _stored(x, transposed, ld=None):
    """The matrix with rows at multiples of 16 bytes, NaN behind them."""
    x = x.t() if transposed else x
    ld = -(-x.shape[1] // 8) * 8 if ld is None else ld
    store = torch.full((x.shape[0], ld), float("nan"), dtype=x.dtype, device=DEV)
    view = store[:, :x.shape[1]]
    view.copy_(x)
    return view


def _in_a_wider_one(rows, cols, dtype, ld, start=0):
    """(buffer, view): a matrix inside a buffer of 7s."""
    store = torch.full((rows + 2, ld), 7.0, dtype=dtype, device=DEV)
    return store, store[1:rows + 1, start:start + cols]


def _only_inside_changed(store, rows, cols, start=0):
    outside = store.clone()
    outside[1:rows + 1, start:start + cols] = 7
    assert bool((outside == 7).all()), "elements outside the matrix changed"


def sum_error(k, size, dtype):
    """What a sum of k products loses, in units of the sum of magnitudes. Every 16 products
    are aligned, with the sum so far, to the largest of the 17 and cut off at 2^-23 of it;
    the parts of split sums add eight roundings at most. fp32 operands: the other five
    products are below 2^-8 of the first, and 2^-23 is left out."""
    steps = -(-k // 16)
    if dtype == FP32:
        return size * (34 * U * steps * (1 + 5 / 256) + 10 * U + 2 * U)
    return size * (34 * U * steps + 10 * U)


def _reference(a, b, bias, act, residual, dtype, out_dtype):
    """(out, bound), (z, bound), bounds before rounding, in 64 bits."""
    a, b = a.double(), b.double()
    z = a @ b.t()
    bz = sum_error(a.shape[1], a.abs() @ b.abs().t(), dtype)
    if bias is not None:
        z = z + bias.double()
        bz = bz + U * (z.abs() + bz)
    if act == "none":
        y, by = z, bz
    elif act == "relu":
        y, by = ref.activation(z, act), bz
    else:
        gate, bg = (z, bz) if act == "gelu" else (z.chunk(2, 1)[0], bz.chunk(2, 1)[0])
        y = gate * ref.phi(gate)
        # |gelu'| < 1.13 everywhere; the argument's error also moves the relative error's z^2.
        by = 1.13 * bg + (ref.phi_error(gate.abs() + bg, out_dtype) + 4 * U) * (y.abs() + bg)
        by = by + ref.TINY * (1 + gate.abs())
        if act == "geglu":
            up, bu = z.chunk(2, 1)[1], bz.chunk(2, 1)[1]
            by = by * (up.abs() + bu) + y.abs() * bu + 2 * U * (y * up).abs()
            y = y * up
    if residual is not None:
        y = y + residual.double()
        by = by + U * (y.abs() + by)
    return (y, by), (z, bz)


def _check(m, n, k, dtype=BF16, out_dtype=None, layout=(False, False), bias=False, act="none",
           residual=False, pre=False, out_ld=None, start=0, seed=61):
    out_dtype = dtype if out_dtype is None else out_dtype
    gen = _gen(seed)
    a = (_randn(gen, m, k) * torch.exp(0.5 * _randn(gen, max(k, 1))[:k])).to(dtype)
    b = (_randn(gen, n, k) / max(k, 1) ** 0.5).to(dtype)
    wide = n // 2 if act == "geglu" else n
    c = (0.3 * _randn(gen, n)).to(out_dtype) if bias else None
    r = _randn(gen, m, wide).to(out_dtype) if residual else None
    ld = wide if out_ld is None else out_ld
    store, out = _in_a_wider_one(m, wide, out_dtype, ld, start)
    pre_ld = n + (ld - wide)
    pre_store, z = _in_a_wider_one(m, n, out_dtype, pre_ld, start) if pre else (None, None)
    got = pe.pe_matmul(_stored(a, layout[0]), _stored(b, layout[1]), bias=c, activation=act,
                       residual=r, out=out, pre=z, a_transposed=layout[0],
                       b_transposed=layout[1])
    assert got is out and pe.pe_read_matmul_status() == 0
    (y, by), (want_z, bz) = _reference(a, b, c, act, r, dtype, out_dtype)
    what = f"{m} x {n} x {k} {act}"
    ref.assert_within(out, y, ref.rounded(by, y, out_dtype), what)
    _only_inside_changed(store, m, wide, start)
    if pre:
        ref.assert_within(z, want_z, ref.rounded(bz, want_z, out_dtype), what + " pre")
        _only_inside_changed(pre_store, m, n, start)
    return out


# Sizes for every way: 16, 32 and 64 rows a CTA without and with a split sum, whole tiles, and
# runs of blocks; ragged in every dimension.
SIZES = [(1, 1, 1), (1, 768, 768), (3, 130, 500), (16, 64, 64), (17, 129, 333), (33, 2304, 768),
         (100, 1001, 1140), (130, 72, 4000), (320, 500, 77), (700, 768, 768), (1537, 768, 320),
         (3001, 1001, 200), (5000, 2304, 96), (300, 300, 20000), (2304, 768, 3000),
         (1000, 1100, 9001)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_of_bf16(m, n, k, layout):
    _check(m, n, k, layout=layout)
    _check(m, n, k, layout=layout, out_dtype=FP32)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_product_of_fp32(m, n, k, layout):
    _check(m, n, k, FP32, layout=layout)


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (BF16, FP32), (FP32, FP32),
                                             (FP32, BF16)])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "geglu"])
@pytest.mark.parametrize("m,n,k", [(1, 768, 768), (5, 200, 64), (50, 514, 900), (200, 1152, 333),
                                   (2000, 2304, 128), (3001, 1000, 130), (300, 300, 12000),
                                   (2304, 770, 4100)])
def test_epilogue(m, n, k, act, dtype, out_dtype):
    _check(m, n, k, dtype, out_dtype, bias=True, act=act, residual=True, pre=True)
    _check(m, n, k, dtype, out_dtype, bias=False, act=act, residual=True, seed=62)
    _check(m, n, k, dtype, out_dtype, bias=True, act=act, pre=True, seed=63)


@pytest.mark.parametrize("out_dtype", [BF16, FP32])
@pytest.mark.parametrize("act", ["none", "geglu"])
@pytest.mark.parametrize("m,n,k", [(3, 128, 128), (2500, 768, 128), (700, 1024, 9000)])
def test_outputs_inside_wider_matrices(m, n, k, act, out_dtype):
    wide = n // 2 if act == "geglu" else n
    for extra, start in ((64, 32), (24, 8), (5, 3), (1, 0)):
        _check(m, n, k, BF16, out_dtype, bias=True, act=act, residual=True, pre=True,
               out_ld=wide + extra, start=start)


@pytest.mark.parametrize("layout", [(False, True), (True, True)])
@pytest.mark.parametrize("m", [5, 3000])
def test_geglu_of_a_transposed_weight(m, layout):
    _check(m, 1040, 300, layout=layout, act="geglu", bias=True, pre=True)
    _check(m, 1040, 300, FP32, layout=layout, act="geglu", bias=True)
    a = _stored(torch.ones(m, 64, device=DEV, dtype=BF16), layout[0])
    b = _stored(torch.ones(24, 64, device=DEV, dtype=BF16), layout[1])
    with pytest.raises(pe.PackedAttentionError, match="status 4"):
        pe.pe_matmul(a, b, activation="geglu", a_transposed=layout[0], b_transposed=layout[1])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("m,n", [(1, 300), (20, 300), (60, 640), (400, 1000), (5000, 777),
                                 (2100, 2100)])
def test_a_permutation_comes_back_exactly(m, n, dtype, layout):
    """b picks columns of a: every bit of every element has to arrive, in its place. fp32
    numbers have all their 24 bits, far from one another in size."""
    gen = _gen(64)
    a = (_randn(gen, m, n) * torch.exp(4 * _randn(gen, m, n))).to(dtype)
    order = torch.randperm(n, generator=gen, device=DEV)
    b = torch.zeros(n, n, dtype=dtype, device=DEV)
    b[torch.arange(n, device=DEV), order] = 1
    got = pe.pe_matmul(_stored(a, layout[0]), _stored(b, layout[1]), a_transposed=layout[0],
                       b_transposed=layout[1])
    assert torch.equal(got, a[:, order])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_empty_sums_and_empty_results(dtype):
    for act in ("none", "gelu", "geglu"):
        _check(5, 64, 0, dtype, bias=True, act=act, residual=True, pre=True)
        _check(700, 514, 0, dtype, bias=True, act=act)
    a, b = torch.ones(0, 64, dtype=dtype, device=DEV), torch.ones(8, 64, dtype=dtype, device=DEV)
    assert pe.pe_matmul(a, b).shape == (0, 8)
    assert pe.pe_matmul(b, a).shape == (8, 0)


@pytest.mark.parametrize("m", [3, 3000])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_infinities_and_nan_stay_in_their_rows(m, dtype):
    gen = _gen(65)
    a, b = _randn(gen, m, 256).to(dtype), _randn(gen, 300, 256).abs().to(dtype) + 0.5
    want = pe.pe_matmul(a, b)
    bad = a.clone()
    bad[1, 7], bad[2, 9] = float("inf"), float("nan")
    got = pe.pe_matmul(bad, b)
    assert bool(got[2].isnan().all())
    assert bool((got[1] == float("inf")).all() if dtype == BF16 else got[1].isnan().all())
    keep = torch.ones(m, dtype=torch.bool, device=DEV)
    keep[1:3] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("m", [2, 3000])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_activations_of_far_and_infinite_sums(m, dtype):
    """The bias is what goes into the activation: gelu and relu at their limits."""
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([-inf, inf, nan, -1e30, 1e30, -70.0, 70.0, -0.0], device=DEV).to(dtype)
    a, b = torch.zeros(m, 64, dtype=dtype, device=DEV), torch.zeros(8, 64, dtype=dtype, device=DEV)
    got = pe.pe_matmul(a, b, bias=z, activation="gelu")
    assert got.nan_to_num(7.0, inf, -inf).double().tolist() == [
        [0.0, inf, 7.0, 0.0, float(z[4]), 0.0, 70.0, 0.0]] * m
    got = pe.pe_matmul(a, b, bias=z, activation="relu")
    assert got.nan_to_num(7.0, inf, -inf).double().tolist() == [
        [0.0, inf, 7.0, 0.0, float(z[4]), 0.0, 70.0, 0.0]] * m
    up = torch.cat([z, torch.ones(8, device=DEV, dtype=dtype)])
    b = torch.zeros(16, 64, dtype=dtype, device=DEV)
    got = pe.pe_matmul(a, b, bias=up, activation="geglu")
    assert got.nan_to_num(7.0, inf, -inf).double().tolist() == [
        [0.0, inf, 7.0, 0.0, float(z[4]), 0.0, 70.0, 0.0]] * m


def test_fp32_numbers_of_all_sizes():
    """Near the largest number, and products far below one another."""
    big = torch.tensor([[3.4028234663852886e38, 1.0, 2.0 ** -60, -3.4e38]], device=DEV)
    pick = torch.eye(4, device=DEV)
    assert torch.equal(pe.pe_matmul(big, pick), big)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("m,n,k", [(3, 200, 100), (3000, 1000, 128), (1000, 768, 6000)])
def test_out_may_be_the_residual(m, n, k, dtype):
    gen = _gen(66)
    a, b, r = (_randn(gen, *s).to(dtype) for s in ((m, k), (n, k), (m, n)))
    a, b = _stored(a, False), _stored(b, False)
    want = pe.pe_matmul(a, b, residual=r)
    into = r.clone()
    assert pe.pe_matmul(a, b, residual=into, out=into) is into
    assert torch.equal(into, want)


def test_operands_that_are_copied_first():
    """Rows that start anywhere, columns that are apart."""
    gen = _gen(67)
    base = _randn(gen, 40, 203).bfloat16()
    b = _randn(gen, 64, 101).bfloat16()
    for a in (base[:, :101], base[:, 2:103], base[:, 1:203:2], base[:1, :101]):
        (y, by), _ = _reference(a, b, None, "none", None, BF16, BF16)
        ref.assert_within(pe.pe_matmul(a, b), y, ref.rounded(by, y, BF16), "copied")


def test_refusals():
    a, b = torch.ones(8, 16, device=DEV), torch.ones(6, 16, device=DEV)
    for bad in (dict(b=b.bfloat16()), dict(b=b[:, :8]), dict(b=b[0]), dict(a=a.double()),
                dict(bias=torch.ones(5, device=DEV)), dict(bias=torch.ones(6, device=DEV).half()),
                dict(residual=a), dict(out=torch.ones(6, 8, device=DEV).t()),
                dict(pre=torch.ones(8, 5, device=DEV)), dict(activation="geglu", b=b[:5]),
                dict(a_transposed=True), dict(dtype=torch.float16),
                dict(out=torch.ones(8, 6)), dict(workspace=torch.ones(1, device=DEV)[:0].cpu())):
        args = dict(a=a, b=b)
        args.update(bad)
        with pytest.raises((ValueError, TypeError)):
            pe.pe_matmul(**args)


WAYS = [(5, 300, 512, BF16), (3, 512, 4000, BF16), (320, 1001, 1140, BF16), (300, 136, 20000, FP32),
        (1537, 768, 1152, BF16), (768, 768, 4504, BF16), (9000, 1152, 768, BF16),
        (9000, 1001, 256, FP32), (2304, 768, 20000, BF16), (2500, 999, 9008, BF16)]


@pytest.mark.parametrize("m,n,k,dtype", WAYS)
def test_runs_are_bitwise_equal_on_any_stream_and_in_graphs(m, n, k, dtype):
    gen = _gen(68)
    a, b, r = (_randn(gen, *s).to(dtype) for s in ((m, k), (n, k), (m, n)))

    def call():
        return pe.pe_matmul(a, b, residual=r)

    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert torch.equal(got, want)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert pe.pe_read_matmul_status() == 0


@pytest.mark.parametrize("m,n,k,dtype", [(5, 304, 512, BF16), (3000, 768, 768, BF16),
                                         (1000, 768, 512, FP32), (2304, 768, 9000, BF16)])
def test_calls_in_turn_read_what_the_one_before_wrote(m, n, k, dtype):
    """The next product may start while the one before still runs; its operand, residual and
    workspace are that one's."""
    gen = _gen(69)
    a, b = _randn(gen, m, k).to(dtype), (_randn(gen, n, k) / k ** 0.5).to(dtype)
    back = (_randn(gen, k, n) / n ** 0.5).to(dtype)
    lib = pe.load_library()
    code = 0 if dtype == BF16 else 1
    need = max(lib.pe_matmul_workspace_size(code, 0, 0, m, n, k, 0),
               lib.pe_matmul_workspace_size(code, 0, 0, m, k, n, 0), 16)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    want, x = [], a
    for _ in range(4):
        y = pe.pe_matmul(x, b)
        torch.cuda.synchronize()
        x = pe.pe_matmul(y, back, residual=x)
        torch.cuda.synchronize()
        want.append((y, x))
    for _ in range(5):
        got, x = [], a
        for _ in range(4):
            y = pe.pe_matmul(x, b, workspace=ws)
            x = pe.pe_matmul(y, back, residual=x, workspace=ws)
            got.append((y, x))
        for (y, x), (wy, wx) in zip(got, want):
            assert torch.equal(y, wy) and torch.equal(x, wx)


# ---------------------------------------------------------------- a layer's step

@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_training_step_of_a_feed_forward_block(dtype):
    """x + dropout(geglu(norm(x) W1^T + b1) W2^T + b2) forwards and backwards by the library's
    calls, its gradients against automatic differentiation in 64 bits."""
    gen = _gen(70)
    n, c, f = 400, 128, 96
    x, dy = _randn(gen, n, c).to(dtype), _randn(gen, n, c).to(dtype)
    w, b = (1 + 0.2 * _randn(gen, c)).to(dtype), (0.1 * _randn(gen, c)).to(dtype)
    w1, b1 = (_randn(gen, 2 * f, c) / c ** 0.5).to(dtype), (0.1 * _randn(gen, 2 * f)).to(dtype)
    w2, b2 = (_randn(gen, c, f) / f ** 0.5).to(dtype), (0.1 * _randn(gen, c)).to(dtype)
    p, seed = 0.25, 77
    h = pe.pe_layernorm(x, w, b)
    z = torch.empty(n, 2 * f, dtype=dtype, device=DEV)
    g = pe.pe_matmul(h, w1, bias=b1, activation="geglu", pre=z)
    u = pe.pe_matmul(g, w2, bias=b2)
    y = pe.pe_dropout(u, p, seed, residual=x)

    du = pe.pe_dropout(dy, p, seed)
    _, db2 = pe.pe_activation_bwd(du, None)
    dw2 = pe.pe_matmul(du, g, dtype=FP32, a_transposed=True, b_transposed=True)
    dg = pe.pe_matmul(du, w2, b_transposed=True)
    dz, db1 = pe.pe_activation_bwd(dg, z, "geglu")
    dw1 = pe.pe_matmul(dz, h, dtype=FP32, a_transposed=True, b_transposed=True)
    dh = pe.pe_matmul(dz, w1, b_transposed=True)
    dx, dw, db = pe.pe_layernorm_bwd(dh, x, w, dresidual=dy)

    leaves = [t.double().requires_grad_() for t in (x, w, b, w1, b1, w2, b2)]
    xd, wd, bd, w1d, b1d, w2d, b2d = leaves
    hd = torch.nn.functional.layer_norm(xd, (c,), wd, bd, 1e-5)
    gate, up = (hd @ w1d.t() + b1d).chunk(2, 1)
    ud = (gate * ref.phi(gate) * up) @ w2d.t() + b2d
    kept = ref.kept(n * c, seed, 0, p).view(n, c).to(DEV)
    yd = xd + torch.where(kept, ud / (1 - p), torch.zeros_like(ud))
    grads = torch.autograd.grad((yd * dy.double()).sum(), leaves)
    # A chain of at most eight results, each rounded to the type and summed over at most 400
    # terms of either sign: 8 half steps of the largest element's size, four times over for the
    # growth of errors through two products whose rows have norm 1 to 2.
    tol = 32 * ref.half_step(dtype) if dtype == BF16 else 3000 * U
    for name, got, want in zip(("y", "x", "w", "b", "w1", "b1", "w2", "b2"),
                               (y, dx, dw, db, dw1, db1, dw2, db2), (yd.detach(), *grads)):
        err = float((got.double() - want).abs().max() / want.abs().max())
        assert err <= tol, f"{name}: {err:.2e}"


@pytest.mark.parametrize("ld", [32768, 32770])
def test_matrices_past_2_to_the_31_elements(ld):
    """Rows that lie far apart: the same numbers as the same matrices without gaps."""
    far, small = 70001, 64
    gen = _gen(61)
    a = torch.empty(far, 32768, dtype=BF16, device=DEV)[:, :small]
    a.copy_(_randn(gen, far, small))
    out = torch.empty(far, ld, dtype=BF16, device=DEV)[:, :small]
    pre = torch.empty(far, ld, dtype=BF16, device=DEV)[:, :small]
    out.copy_(_randn(gen, far, small))
    b = _randn(gen, small, small).bfloat16()
    tight, tight_pre, near = a.contiguous(), torch.empty(far, small, dtype=BF16, device=DEV), \
        out.contiguous()
    want = pe.pe_matmul(tight, b, activation="relu", residual=near, pre=tight_pre)
    pe.pe_matmul(a, b, activation="relu", residual=out, pre=pre, out=out)
    assert torch.equal(out, want) and torch.equal(pre, tight_pre)
    # The same rows as b of a product with few rows, and as both operands of a long sum.
    x = _randn(gen, 3, small).bfloat16()
    assert torch.equal(pe.pe_matmul(x, a), pe.pe_matmul(x, tight))
    both = dict(dtype=FP32, a_transposed=True, b_transposed=True)
    assert torch.equal(pe.pe_matmul(a, a, **both), pe.pe_matmul(tight, tight, **both))


@pytest.mark.parametrize("m", [1, 2, 3, 4, 9, 64])
@pytest.mark.parametrize("n,k", [(1, 3), (7, 130), (96, 768), (33, 1001), (64, 4100)])
@pytest.mark.parametrize("act", ["none", "geglu"])
def test_few_products_of_fp32(m, n, k, act):
    """Rows by fours and what is left of them, one to eight warps a column, a last piece of k
    of one to three elements; results in both types, inside wider matrices."""
    n += n % 2 if act == "geglu" else 0
    for out_dtype in (FP32, BF16):
        _check(m, n, k, dtype=FP32, out_dtype=out_dtype, bias=True, act=act, residual=True,
               pre=True, out_ld=(n // 2 if act == "geglu" else n) + 5)


def test_few_products_of_rows_that_start_anywhere():
    gen = _gen(67)
    a, b = _randn(gen, 3, 66), _randn(gen, 40, 71)
    want = pe.pe_matmul(a[:, 1:65].contiguous(), b[:, 3:67].contiguous())
    got = pe.pe_matmul(a[:, 1:65], b[:, 3:67])
    z = a[:, 1:65].double() @ b[:, 3:67].double().t()
    bound = sum_error(64, a[:, 1:65].double().abs() @ b[:, 3:67].double().abs().t(), FP32)
    ref.assert_within(got, z, ref.rounded(bound, z, FP32), "odd rows")
    ref.assert_within(want, z, ref.rounded(bound, z, FP32), "the same, aligned")
