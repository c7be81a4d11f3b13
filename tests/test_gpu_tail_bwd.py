"""The layer tail's backward calls, dropout and rotary positions with several axes on the GPU
against their definitions in 64 bits."""

import pytest
import torch

import padding_free_packed_gb300 as pe
import tail_reference as ref
from tail_reference import U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
DTYPES = [BF16, FP32]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _shifted(t, by):
    """The same values in a buffer that starts `by` elements later."""
    store = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    view = store[by:].view(t.shape)
    view.copy_(t)
    return view


# ---------------------------------------------------------------- LayerNorm backward

def _check_layernorm_bwd(n, c, dtype, dres, seed=1, mean=0.0, **kw):
    gen = _gen(seed)
    h = ((_randn(gen, n, c) + mean) * torch.exp(0.5 * _randn(gen, c))).to(dtype)
    dy = _randn(gen, n, c).to(dtype)
    w = (1 + 0.3 * _randn(gen, c)).to(dtype)
    r = _randn(gen, n, c).to(dtype) if dres else None
    dx, dw, db = pe.pe_layernorm_bwd(dy, h, w, 1e-5, dresidual=r, **kw)
    (want, bound), (want_w, terms, term_err), want_b = ref.layernorm_bwd(
        dy.double(), h.double(), w.double(), 1e-5, None if r is None else r.double())
    ref.assert_within(dx, want, ref.rounded(bound, want, dtype), f"dx {n} x {c}")
    # A thread adds at most ceil(n / 152) rows one after the other (456 blocks, 152 for wide
    # rows), eight groups, 32 threads' lines of 456 / 32, and 5 steps of a warp.
    depth = (-(-n // 152) + 8 + 15 + 5 + 4) * U
    ref.assert_within(dw, want_w, term_err + depth * terms + 1e-38, f"dweight {n} x {c}")
    ref.assert_within(db, want_b, depth * dy.double().abs().sum(0) + 1e-38, f"dbias {n} x {c}")
    return dx, dw, db


WIDTHS = [1, 2, 7, 8, 63, 64, 129, 255, 256, 257, 333, 500, 512, 768, 1000, 1024, 1140, 2048, 2304,
          2305, 4096, 4097, 9001, 16384]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("c", WIDTHS)
@pytest.mark.parametrize("dres", [False, True])
def test_layernorm_bwd(c, dtype, dres):
    _check_layernorm_bwd(37 if c > 600 else 301, c, dtype, dres)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,c", [(1, 768), (2, 333), (20011, 256), (20011, 250), (9001, 512),
                                 (9001, 768), (5003, 1001), (5003, 1536), (2503, 4100),
                                 (1001, 8192)])
def test_layernorm_bwd_of_many_rows(n, c, dtype):
    _check_layernorm_bwd(n, c, dtype, True, seed=2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,c", [(193, 520), (300, 768), (193, 776), (2000, 1024), (97, 1028),
                                 (700, 1040), (700, 1536), (700, 1544), (49, 2304), (700, 2304),
                                 (700, 2312), (49, 4096), (461, 4096)])
def test_layernorm_bwd_of_rows_in_shared_memory(n, c, dtype):
    """Rows wide enough to wait in shared memory, from one more than one launch takes to
    several a group of threads, with and without the residual's gradient, and in place."""
    _check_layernorm_bwd(n, c, dtype, False, seed=7)
    want = _check_layernorm_bwd(n, c, dtype, True, seed=8)
    gen = _gen(8)
    h = (_randn(gen, n, c) * torch.exp(0.5 * _randn(gen, c))).to(dtype)
    dy = _randn(gen, n, c).to(dtype)
    w = (1 + 0.3 * _randn(gen, c)).to(dtype)
    r = _randn(gen, n, c).to(dtype)
    for which in range(3):
        t = [dy.clone(), h.clone(), r.clone()]
        got = pe.pe_layernorm_bwd(t[0], t[1], w, 1e-5, dresidual=t[2], out=t[which])
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", DTYPES)
def test_layernorm_bwd_with_a_large_mean(dtype):
    _check_layernorm_bwd(300, 768, dtype, False, seed=3, mean=100.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_layernorm_bwd_in_place_and_no_rows(dtype):
    gen = _gen(4)
    h, dy, r = (_randn(gen, 77, 500).to(dtype) for _ in range(3))
    w = _randn(gen, 500).to(dtype)
    want = pe.pe_layernorm_bwd(dy, h, w, dresidual=r)
    for which in range(3):
        t = [dy.clone(), h.clone(), r.clone()]
        got = pe.pe_layernorm_bwd(t[0], t[1], w, dresidual=t[2], out=t[which])
        assert got[0].data_ptr() == t[which].data_ptr()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    dx, dw, db = pe.pe_layernorm_bwd(dy[:0], h[:0], w)
    assert dx.shape == (0, 500) and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_layernorm_bwd_of_a_constant_row(dtype):
    """A row without variance: n is 0, rstd 1 / sqrt(eps)."""
    h = torch.full((3, 64), 2.0, dtype=dtype, device=DEV)
    dy = _randn(_gen(5), 3, 64).to(dtype)
    w = torch.ones(64, dtype=dtype, device=DEV)
    dx, dw, _ = pe.pe_layernorm_bwd(dy, h, w, 1e-2)
    want = (dy.double() - dy.double().mean(1, keepdim=True)) * 10
    ref.assert_within(dx, want, ref.rounded(64 * U * 20 * dy.double().abs().amax(), want, dtype),
                      "dx")
    assert not dw.any()


def test_layernorm_bwd_against_differences():
    """The gradient of sum(y * dy) by central differences of the definition in 64 bits."""
    gen = _gen(6)
    h, dy, w = _randn(gen, 5, 24), _randn(gen, 5, 24), _randn(gen, 24)
    dx, dw, db = pe.pe_layernorm_bwd(dy, h, w)

    def loss(hh, ww):
        d = hh - hh.mean(1, keepdim=True)
        y = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * ww
        return (y * dy.double()).sum()

    step = 1e-5
    for i in range(24):
        e = torch.zeros(24, dtype=torch.float64, device=DEV)
        e[i] = step
        row = torch.zeros(5, 24, dtype=torch.float64, device=DEV)
        row[2, i] = step
        hd, wd = h.double(), w.double()
        assert abs(float((loss(hd + row, wd) - loss(hd - row, wd)) / (2 * step) - dx[2, i])) < 1e-4
        assert abs(float((loss(hd, wd + e) - loss(hd, wd - e)) / (2 * step) - dw[i])) < 1e-4


# ---------------------------------------------------------------- activation backward

ACTS = ["none", "relu", "gelu", "geglu"]


def _check_activation_bwd(n, f, act, dtype, seed=11, scale=2.0, shift=0):
    gen = _gen(seed)
    dy = _shifted(_randn(gen, n, f).to(dtype), shift)
    z = None
    if act != "none":
        z = _shifted((scale * _randn(gen, n, 2 * f if act == "geglu" else f)).to(dtype), shift)
    dz, db = pe.pe_activation_bwd(dy, z, act)
    want, bound = ref.activation_bwd(dy.double(), None if z is None else z.double(), act, dtype)
    what = f"{act} {n} x {f}"
    ref.assert_within(dz, want, ref.rounded(bound, want, dtype) if act != "none" else 0 * want,
                      what)
    # A thread adds its rows one after the other: 16 a block and at least one block for every
    # 8 x 152 / strips, strips of 16 columns at least.
    lines = max(1, min(304, -(-n // 16), 8 * 152 // -(-f // 16)))
    depth = (-(-n // (16 * lines)) + 16 + 10 + 5 + 4) * U
    ref.assert_within(db, want.sum(0), bound.sum(0) + depth * (want.abs() + bound).sum(0) + 1e-38,
                      what + " dbias")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n,f", [(1, 1), (1, 768), (3, 7), (301, 64), (301, 333), (1001, 500),
                                 (257, 1152), (33, 2305), (20011, 130)])
def test_activation_bwd(n, f, act, dtype):
    _check_activation_bwd(n, f, act, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
def test_activation_bwd_from_any_element(act, dtype):
    _check_activation_bwd(130, 256, act, dtype, shift=1)
    _check_activation_bwd(130, 256, act, dtype, shift=2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["gelu", "geglu"])
def test_activation_bwd_far_arguments(act, dtype):
    """Gates far on both sides, where gelu's tail decides."""
    _check_activation_bwd(512, 128, act, dtype, seed=12, scale=6.0)
    z = torch.tensor([[-1e30, -50.0, -0.0, 0.0, 50.0, 1e30]], device=DEV).to(dtype)
    dy = torch.ones_like(z)
    dz, _ = pe.pe_activation_bwd(dy, z, "gelu")
    assert dz.tolist() == [[0.0, 0.0, 0.5, 0.5, 1.0, 1.0]]
    inf = float("inf")
    z = torch.tensor([[-inf, inf, float("nan")] * 2], device=DEV).to(dtype)
    dz, _ = pe.pe_activation_bwd(torch.ones(1, 6 if act == "gelu" else 3, device=DEV).to(dtype), z,
                                 act)
    if act == "gelu":
        assert dz[0, :2].tolist() == [0.0, 1.0] and bool(dz[0, 2].isnan())
    else:                                       # gate and up are both (-inf, inf, nan)
        assert dz[0, 3:5].tolist() == [0.0, inf] and bool(dz[0, 5].isnan())


@pytest.mark.parametrize("dtype", DTYPES)
def test_activation_bwd_in_place_and_no_rows(dtype):
    gen = _gen(13)
    dy, z, wide = (_randn(gen, 61, w).to(dtype) for w in (100, 100, 200))
    for act, pre in (("relu", z), ("gelu", z), ("geglu", wide)):
        want, sums = pe.pe_activation_bwd(dy, pre, act)
        into = pre.clone()
        got, again = pe.pe_activation_bwd(dy, into, act, out=into)
        assert torch.equal(got, want) and torch.equal(again, sums)
        if act != "geglu":
            into = dy.clone()
            got, _ = pe.pe_activation_bwd(into, pre, act, out=into)
            assert torch.equal(got, want)
        got, none = pe.pe_activation_bwd(dy, pre, act, need_dbias=False)
        assert none is None and torch.equal(got, want)
        got, sums = pe.pe_activation_bwd(dy[:0], pre[:0], act)
        assert got.shape == (0, pre.shape[1]) and not sums.any()


def test_geglu_backward_against_differences():
    gen = _gen(14)
    dy, z = _randn(gen, 3, 9), _randn(gen, 3, 18)
    dz, db = pe.pe_activation_bwd(dy, z, "geglu")
    step = 1e-5
    for i in range(18):
        e = torch.zeros(3, 18, dtype=torch.float64, device=DEV)
        e[1, i] = step
        up = (ref.activation(z.double() + e, "geglu") * dy.double()).sum()
        down = (ref.activation(z.double() - e, "geglu") * dy.double()).sum()
        assert abs(float((up - down) / (2 * step) - dz[1, i])) < 1e-4


# ---------------------------------------------------------------- dropout

def _check_dropout(x, p, seed, offset, residual=None):
    y = pe.pe_dropout(x, p, seed, offset, residual=residual)
    kept = ref.kept(x.numel(), seed, offset, p).view(x.shape).to(DEV)
    want = torch.where(kept, x.double() / (1 - p), 0.0)
    bound = 2 * U * want.abs()                       # the factor and the product
    if residual is not None:
        want = want + residual.double()
        bound = bound + U * want.abs()
    ref.assert_within(y, want, ref.rounded(bound, want, x.dtype), f"{tuple(x.shape)} p {p}")
    return y, kept


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1,), (3,), (5, 7), (1, 768), (33, 500), (64, 129)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(shape, p, dtype, residual):
    gen = _gen(21)
    x = _randn(gen, *shape).to(dtype)
    r = _randn(gen, *shape).to(dtype) if residual else None
    _check_dropout(x, p, 2 ** 63 + 12345, 2 ** 40 + 3, r)


@pytest.mark.parametrize("dtype", DTYPES)
def test_dropout_mask_depends_on_the_numbers_alone(dtype):
    """The same mask for every type, alignment and direction; another for another offset."""
    gen = _gen(22)
    x = _randn(gen, 1003).to(dtype) + 3
    y, kept = _check_dropout(x, 0.4, 7, 0)
    shifted = _shifted(x, 1)
    assert torch.equal(pe.pe_dropout(shifted, 0.4, 7), y)
    assert torch.equal(pe.pe_dropout(torch.ones_like(x), 0.4, 7) != 0, kept)
    other = pe.pe_dropout(x, 0.4, 7, 1)
    assert not torch.equal(other, y)
    assert not torch.equal(pe.pe_dropout(x, 0.4, 8), y)
    one = torch.ones(1, dtype=torch.int64, device=DEV)
    assert torch.equal(pe.pe_dropout(x, 0.4, 7, device_offset=one), other)
    assert torch.equal(pe.pe_dropout(x, 0.4, 7, 2 ** 64 - 1, device_offset=one), y)


def test_dropout_drops_infinities_and_keeps_the_share():
    x = torch.full((1 << 20,), float("inf"), device=DEV)
    y = pe.pe_dropout(x, 0.25, 99)
    assert bool(((y == 0) | (y == float("inf"))).all())
    share = float((y == 0).double().mean())
    assert abs(share - 0.25) < 6 * (0.25 * 0.75 / 2 ** 20) ** 0.5      # six deviations
    y = pe.pe_dropout(x, 1 - 2.0 ** -40, 99)                           # threshold 2^32: none kept
    assert not y.any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_dropout_in_place_and_empty(dtype):
    gen = _gen(23)
    x, r = _randn(gen, 4097).to(dtype), _randn(gen, 4097).to(dtype)
    want = pe.pe_dropout(x, 0.3, 5, residual=r)
    a, b = x.clone(), r.clone()
    assert torch.equal(pe.pe_dropout(a, 0.3, 5, residual=r, out=a), want)
    assert torch.equal(pe.pe_dropout(x, 0.3, 5, residual=b, out=b), want)
    assert pe.pe_dropout(x[:0], 0.3, 5).shape == (0,)


def test_dropout_of_a_captured_graph_draws_anew():
    x = _randn(_gen(24), 5000)
    counter = torch.zeros(1, dtype=torch.int64, device=DEV)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pe.pe_dropout(x, 0.5, 11, 100, device_offset=counter, out=out)
    for i in range(3):
        counter.fill_(i)
        graph.replay()
        assert torch.equal(out, pe.pe_dropout(x, 0.5, 11, 100 + i))


# ---------------------------------------------------------------- rotary positions

def _qkv(gen, n, heads, d, dtype, fused):
    if fused:
        qkv = _randn(gen, n, 3, heads, d).to(dtype)
        return qkv[:, 0], qkv[:, 1]
    return _randn(gen, n, heads, d).to(dtype), _randn(gen, n, max(heads // 2, 1), d).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,d,sections", [
    (1, 2, (1,)), (2, 64, (32,)), (12, 64, (16, 16)), (8, 64, (8, 12, 12)), (3, 40, (5, 15)),
    (4, 72, (12, 12, 12)), (16, 128, (16, 24, 24)), (2, 256, (32, 32, 32, 32)),
    (5, 18, (0, 4, 5)), (9, 66, (33,))])
@pytest.mark.parametrize("per_axis", [False, True])
@pytest.mark.parametrize("fused", [False, True])
def test_rope_axes(heads, d, sections, per_axis, dtype, fused):
    gen = _gen(31)
    for n in (1, 7, 300):
        q, k = _qkv(gen, n, heads, d, dtype, fused)
        pos = torch.randint(-50, 9000, (len(sections), n), generator=gen, device=DEV,
                            dtype=torch.int32)
        for inverse in (False, True):
            got = pe.pe_rope_axes(q, k, pos, sections, 10000.0, per_axis=per_axis,
                                  inverse=inverse)
            angles = ref.rope_angles(pos, sections, 10000.0, per_axis) * (-1 if inverse else 1)
            for x, y in zip((q, k), got):
                want, bound = ref.rope(x.double(), angles)
                ref.assert_within(y, want, ref.rounded(bound, want, dtype),
                                  f"{n} {heads} x {d} {sections}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_rope_axes_at_the_ends_of_int32(dtype):
    """Positions whose angles are billions of turns; the reference's own angles, of two fp32
    halves of exact products, keep 2^-52 of at most 2^31 radians, 5e-7."""
    gen = _gen(32)
    pos = torch.tensor([[-2 ** 31, 2 ** 31 - 1, 0, 1, -1, 123456789]], dtype=torch.int32,
                       device=DEV)
    q = _randn(gen, 6, 2, 64).to(dtype)
    got, _ = pe.pe_rope_axes(q, None, pos, (32,), 10000.0)
    angles = ref.rope_angles(pos, (32,), 10000.0, False)
    want, bound = ref.rope(q.double(), angles)
    size = q.double().abs().amax()
    # theta^(-2i/D) itself carries 2^-53 on either side: 2^31 radians times 2^-51.
    ref.assert_within(got, want, ref.rounded(bound + 2 * size * 2.0 ** -20, want, dtype), "far")


@pytest.mark.parametrize("dtype", DTYPES)
def test_rope_axes_is_rope_packed_for_one_axis(dtype):
    gen = _gen(33)
    q, k = _qkv(gen, 200, 4, 64, dtype, False)
    pos = torch.randint(0, 8192, (200,), generator=gen, device=DEV, dtype=torch.int32)
    got_q, got_k = pe.pe_rope_axes(q, k, pos[None], (32,), 160000.0)
    pe.pe_rope_packed(q, k, pos, 160000.0)
    for got, want in ((got_q, q), (got_k, k)):
        step = 2 * ref.half_step(dtype) * want.double().abs() + 16 * U * 6   # |x1| + |x2| < 12
        ref.assert_within(got, want, step, "one axis")


@pytest.mark.parametrize("dtype", DTYPES)
def test_rope_axes_in_place_and_into_views(dtype):
    gen = _gen(34)
    qkv = _randn(gen, 130, 3, 6, 40).to(dtype)
    before = qkv.clone()
    pos = torch.randint(0, 256, (2, 130), generator=gen, device=DEV, dtype=torch.int32)
    want_q, want_k = pe.pe_rope_axes(qkv[:, 0], qkv[:, 1], pos, (10, 10), 1e4, per_axis=True)
    assert want_q.is_contiguous() and want_k.is_contiguous()
    assert torch.equal(qkv, before)
    pe.pe_rope_axes(qkv[:, 0], qkv[:, 1], pos, (10, 10), 1e4, per_axis=True, out_q=qkv[:, 0],
                    out_k=qkv[:, 1])
    assert torch.equal(qkv[:, 0], want_q) and torch.equal(qkv[:, 1], want_k)
    assert torch.equal(qkv[:, 2], before[:, 2])
    back = torch.full((130, 2, 6, 40), 7.0, dtype=dtype, device=DEV)
    pe.pe_rope_axes(want_q, None, pos, (10, 10), 1e4, per_axis=True, inverse=True,
                    out_q=back[:, 1])
    assert bool((back[:, 0] == 7).all())
    size = 2 * before[:, 0].double().abs().amax()
    ref.assert_within(back[:, 1], before[:, 0].double(),
                      (3 * ref.half_step(dtype) + 32 * U) * size + 0 * back[:, 1].double(), "back")


def test_rope_axes_refusals():
    q = torch.zeros(4, 2, 8, device=DEV)
    pos = torch.zeros(2, 4, dtype=torch.int32, device=DEV)
    for bad in (dict(positions=pos.long()), dict(positions=pos[:1]), dict(sections=(2, 2, 0)),
                dict(q=q.transpose(1, 2)), dict(q=q[0]), dict(k=q[:3]), dict(k=q.bfloat16()),
                dict(out_q=q[:3]), dict(out_q=q.double()), dict(k=None, out_k=q)):
        args = dict(q=q, k=q, positions=pos, sections=(2, 2), theta=1e4)
        args.update(bad)
        with pytest.raises(ValueError):
            pe.pe_rope_axes(**args)
    with pytest.raises(pe.PackedAttentionError):
        pe.pe_rope_axes(q, q, pos, (2, 3), 1e4)
    with pytest.raises(pe.PackedAttentionError):
        pe.pe_rope_axes(q[:, :, :7].contiguous(), None, pos, (2, 1), 1e4)


# ---------------------------------------------------------------- all calls

def _calls():
    gen = _gen(41)
    h, dy, r = (_randn(gen, 300, 256).bfloat16() for _ in range(3))
    w = _randn(gen, 256).bfloat16()
    z = _randn(gen, 300, 512).bfloat16()
    pos = torch.randint(0, 99, (2, 300), generator=gen, device=DEV, dtype=torch.int32)
    return [lambda: pe.pe_layernorm_bwd(dy, h, w, dresidual=r),
            lambda: pe.pe_activation_bwd(dy, z, "geglu"),
            lambda: [pe.pe_dropout(h, 0.2, 3, residual=r)],
            lambda: pe.pe_rope_axes(h.view(300, 4, 64), r.view(300, 4, 64), pos, (16, 16), 1e4)]


@pytest.mark.parametrize("which", range(4))
def test_runs_are_bitwise_equal_on_any_stream_and_in_graphs(which):
    call = _calls()[which]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for _ in range(2):                               # two graphs, each with its own workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_layernorm_bwd_by_two_launches_in_two_graphs_at_a_time():
    gen = _gen(41)
    h, dy, r = (_randn(gen, 2000, 1024).bfloat16() for _ in range(3))
    w = _randn(gen, 1024).bfloat16()
    want = [t.clone() for t in pe.pe_layernorm_bwd(dy, h, w, dresidual=r)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(pe.pe_layernorm_bwd(dy, h, w, dresidual=r))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


# ---------------------------------------------------------------- offsets past 32 bits

def test_rows_past_2_to_the_31_elements():
    """The last rows are those that a call on them alone gives: dx, dz and a dropout's elements
    depend on nothing else (a dropout's on their index, which the definition counts in 64
    bits)."""
    c, n, tail = 1024, (1 << 21) + 300, 300
    gen = _gen(42)
    dy, h = (torch.empty(n, c, dtype=BF16, device=DEV).normal_(generator=gen) for _ in range(2))
    w = _randn(gen, c).bfloat16()
    dx = pe.pe_layernorm_bwd(dy, h, w)[0]
    want = pe.pe_layernorm_bwd(dy[-tail:], h[-tail:], w)[0]
    assert torch.equal(dx[-tail:], want)
    del dx
    dz, _ = pe.pe_activation_bwd(dy, h, "gelu")
    assert torch.equal(dz[-tail:], pe.pe_activation_bwd(dy[-tail:], h[-tail:], "gelu")[0])
    del dz
    y = pe.pe_dropout(h, 0.3, 5, 6)
    words = [w for block in range((n - 1) * c // 4, n * c // 4)
             for w in ref.philox_words(block, 5, 6)]
    kept = torch.tensor([word >= 0.3 * 2 ** 32 for word in words], device=DEV)
    x = h[-1].double()
    want = torch.where(kept, x / 0.7, 0.0)
    ref.assert_within(y[-1], want, ref.rounded(2 * U * want.abs(), want, BF16), "dropout")


def test_rope_of_tokens_past_2_to_the_31_elements():
    n, step, tail = 70001, 32768, 50
    store = torch.empty(n, step, dtype=BF16, device=DEV).normal_(generator=_gen(43))
    q, k = store[:, :512].view(n, 8, 64), store[:, 1024:1280].view(n, 4, 64)
    pos = torch.randint(0, 1 << 20, (2, n), dtype=torch.int32, device=DEV, generator=_gen(44))
    want = pe.pe_rope_axes(q[-tail:].contiguous(), k[-tail:].contiguous(), pos[:, -tail:],
                           (12, 20), 1e4)
    untouched = store[-tail:, 512:1024].clone()
    got = pe.pe_rope_axes(q, k, pos, (12, 20), 1e4, out_q=q, out_k=k)
    for a, b in zip(got, want):
        assert torch.equal(a[-tail:], b)
    assert torch.equal(store[-tail:, 512:1024], untouched)


def test_rope_refuses_sections_that_32_bits_do_not_hold():
    q = torch.zeros(2, 1, 64, device=DEV)
    pos = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        pe.pe_rope_axes(q, None, pos, (2 ** 32 + 32,), 1e4)
