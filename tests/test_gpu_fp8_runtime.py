"""The 8-bit layer calls as a program meets them: waits that give up, graphs,
streams, buffers of any alignment, sizes past 32 bits, and refused tensors."""

import os
import subprocess
import sys

import pytest
import torch

import fp8_reference as ref
import padding_free_packed_gb300 as pe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
BF16, FP32 = torch.bfloat16, torch.float32
TIMEOUT = 7
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def _product(seed, m, n, k):
    return (*pe.pe_quantize_fp8(_randn(seed, m, k)), *pe.pe_quantize_fp8(_randn(seed + 1, n, k), 128))


# One of every way a product runs: narrow tiles without and with a shared sum, pairs
# on whole tiles with each form of output, pairs on shared tiles.
WAYS = [(5, 300, 500, BF16), (3, 512, 4000, BF16), (60, 200, 9000, FP32), (9000, 1024, 768, BF16),
        (9000, 1024, 768, FP32), (9000, 1001, 768, BF16), (2304, 768, 20000, FP32),
        (2304, 999, 20000, BF16)]


@pytest.mark.parametrize("m,n,k,dtype", WAYS)
def test_wait_timeout_is_reported_and_the_next_call_is_correct(m, n, k, dtype):
    """With a 1 ns limit the waits give up and the status word says so, once; with
    the default limit the next call equals the one before."""
    ops = _product(401, m, n, k)
    want = pe.pe_matmul_fp8(*ops, dtype=dtype)
    assert pe.pe_read_matmul_status() == 0
    previous = pe.pe_set_wait_limit_ns(1)
    try:
        for _ in range(3):
            pe.pe_matmul_fp8(*ops, dtype=dtype)
        assert pe.pe_read_matmul_status() == TIMEOUT
        assert pe.pe_read_matmul_status() == 0                   # read and cleared
    finally:
        pe.pe_set_wait_limit_ns(previous)
    assert torch.equal(pe.pe_matmul_fp8(*ops, dtype=dtype), want)
    assert pe.pe_read_matmul_status() == 0


@pytest.mark.parametrize("limit_ns", [300, 2000, 20000])
@pytest.mark.parametrize("m,n,k", [(9000, 1024, 768), (2304, 768, 9000)])
def test_wait_limits_near_the_waits_themselves(m, n, k, limit_ns):
    """Limits that some waits exceed and others do not, so that a pair's CTAs give
    up at different blocks: the status tells, and no later call suffers."""
    ops = _product(402, m, n, k)
    want = pe.pe_matmul_fp8(*ops)
    previous = pe.pe_set_wait_limit_ns(limit_ns)
    try:
        for _ in range(3):
            got = pe.pe_matmul_fp8(*ops)
            assert pe.pe_read_matmul_status() in (0, TIMEOUT)
    finally:
        pe.pe_set_wait_limit_ns(previous)
    got = pe.pe_matmul_fp8(*ops)
    assert pe.pe_read_matmul_status() == 0
    assert torch.equal(got, want)


FIRST_CALL_IN_A_GRAPH = r"""
import torch
import padding_free_packed_gb300 as pe
x = torch.ones(300, 256, device="cuda", dtype=torch.bfloat16)
w = torch.ones(256, device="cuda", dtype=torch.bfloat16)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    q, s = pe.pe_rmsnorm_fp8(x, w)
    wq, ws = pe.pe_quantize_fp8(x[:200], 128)
    out = pe.pe_matmul_fp8(q, s, wq, ws)
    big = pe.pe_matmul_fp8(*pe.pe_quantize_fp8(torch.ones(9000, 256, device="cuda")), wq, ws)
    dx, dw = pe.pe_rmsnorm_bwd(out.new_ones(300, 256), x, w)
graph.replay()
torch.cuda.synchronize()
assert out.shape == (300, 200) and float(out.float().min()) == float(out.float().max()) == 256.0
assert float(big.float().min()) == float(big.float().max()) == 256.0
assert float(dw.min()) == float(dw.max()) and abs(float(dw[0]) - 300) < 0.01
print("replayed")
"""


def test_a_process_whose_first_calls_are_captured():
    """Nothing needs a call before the capture: ones times ones, exact in 8 bits
    (the norm of ones with eps 1e-5 quantises to its block's largest value, and the
    scale brings back 1 - 5e-6, which is 1 in the bf16 product)."""
    run = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_GRAPH], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "replayed" in run.stdout, run.stderr[-2000:]


def test_two_graphs_replayed_in_turn_and_at_once():
    """Graphs hold workspaces of their own; replayed on two streams together they
    give what they give alone."""
    sets = [_product(410 + i, 2304, 768, 9000) for i in range(2)]
    norms = [(_randn(420 + i, 5000, 768).to(BF16), _randn(430 + i, 5000, 768).to(BF16),
              _randn(440 + i, 768).to(BF16)) for i in range(2)]

    def step(i):
        return (pe.pe_matmul_fp8(*sets[i], dtype=FP32), *pe.pe_rmsnorm_bwd(*norms[i]))

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(i))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for together in (False, True):
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
                if not together:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        for i in range(2):
            for got, one in zip(outs[i], want[i]):
                assert torch.equal(got, one)


def test_a_workspace_of_the_caller():
    ops = _product(450, 2304, 768, 9000)
    want = pe.pe_matmul_fp8(*ops)
    need = pe.load_library().pe_matmul_fp8_workspace_size(2304, 768, 9000)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)      # NaN in every word
    for _ in range(2):
        assert torch.equal(pe.pe_matmul_fp8(*ops, workspace=ws), want)
    with pytest.raises(pe.PackedAttentionError) as e:
        pe.pe_matmul_fp8(*ops, workspace=ws[:-1])
    assert e.value.status == 5
    dy, h, w = _randn(451, 700, 333), _randn(452, 700, 333), _randn(453, 333)
    dx, dw = pe.pe_rmsnorm_bwd(dy, h, w)
    need = pe.load_library().pe_rmsnorm_bwd_workspace_size(333)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    got = pe.pe_rmsnorm_bwd(dy, h, w, workspace=ws)
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)


def _shifted(t, elements=1):
    """The same values at an address `elements` further than a fresh allocation."""
    flat = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)[elements:]
    return flat.view(t.shape).copy_(t)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("c", [256, 768])
def test_buffers_of_any_alignment(dtype, c):
    """Tensors one element past a 16-byte boundary. The vector and the element-wise
    kernels add a row in different orders, so norms agree to their error bound and
    quantised tensors, whose maxima have no order, are equal."""
    x, r, w = (_randn(460 + i, *s).to(dtype) for i, s in enumerate([(130, c), (130, c), (c,)]))
    xs, rs, wsh = _shifted(x), _shifted(r), _shifted(w)
    y, h = pe.pe_rmsnorm(xs, wsh, residual=rs, out=_shifted(x), residual_out=_shifted(x))
    want, want_h = ref.rmsnorm(x, w, 1e-5, r)
    assert torch.equal(h, want_h)
    rel = ref.rmsnorm_rel(c)
    assert bool(((y.double() - want).abs() <= (rel + ref.half_step(dtype) + rel) * want.abs()
                 + 1e-38).all())
    q, s, _ = pe.pe_rmsnorm_fp8(xs, wsh, residual=rs)
    ref.check_quantized(q, s, want, E4M3, 1, rel, "norm")
    for got, one in zip(pe.pe_quantize_fp8(xs, 1, transposed=True),
                        pe.pe_quantize_fp8(x, 1, transposed=True)):
        assert torch.equal(got.float(), one.float())
    dx, dw = pe.pe_rmsnorm_bwd(xs, rs, wsh, dresidual=_shifted(r), out=_shifted(x))
    want_dx, want_dw, size, dw_size = ref.rmsnorm_bwd(x, r, w, 1e-5, r)
    bound = (2.5 * ref.norm_depth(c) + 24) * ref.U * size + ref.half_step(dtype) * want_dx.abs() * (
        1 + 2 ** -8)
    assert bool(((dx.double() - want_dx).abs() <= bound).all())
    ops = _product(465, 300, c, 256)
    out = _shifted(torch.empty(300, c, dtype=dtype, device=DEV))
    assert torch.equal(pe.pe_matmul_fp8(*ops, out=out), pe.pe_matmul_fp8(*ops, dtype=dtype))
    ops = _product(466, 9000, c, 256)
    out = _shifted(torch.empty(9000, c, dtype=dtype, device=DEV))
    assert torch.equal(pe.pe_matmul_fp8(*ops, out=out), pe.pe_matmul_fp8(*ops, dtype=dtype))


def test_one_matrix_as_both_operands():
    x = _randn(470, 1000, 500)
    q, s = pe.pe_quantize_fp8(x, 1)
    sq, ss = pe.pe_quantize_fp8(x, 128)
    mixed = pe.pe_matmul_fp8(q, s, sq, ss, dtype=FP32)
    want, size = ref.matmul(q, s, sq, ss)
    assert bool(((mixed.double() - want).abs() <= ref.matmul_rel(500) * size).all())
    spread = ss.repeat_interleave(128, 1)[:, :1000].contiguous()  # the same scales, row by row
    both = pe.pe_matmul_fp8(sq, spread, sq, ss, dtype=FP32)
    assert torch.equal(both, both.t())


def test_on_another_stream_than_the_default():
    stream = torch.cuda.Stream()
    x, w = _randn(480, 4000, 768).to(BF16), _randn(481, 768).to(BF16)
    wq = pe.pe_quantize_fp8(_randn(482, 512, 768), 128)
    want = pe.pe_matmul_fp8(*pe.pe_rmsnorm_fp8(x, w), *wq)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        late = torch.zeros_like(x)
        torch.cuda._sleep(20_000_000)
        late.copy_(x)                                  # after the wait, on this stream
        got = pe.pe_matmul_fp8(*pe.pe_rmsnorm_fp8(late, w), *wq)
    stream.synchronize()
    assert torch.equal(got, want)


def test_more_than_two_to_the_31_elements():
    """Element offsets past 32 bits: the last rows of a large call equal a small
    call on those rows alone."""
    n, c, tail = (1 << 21) + 131, 1030, 259                    # 2.16e9 elements
    x = torch.empty(n, c, dtype=BF16, device=DEV)
    for part in x.split(1 << 18):
        part.normal_()
    w = _randn(491, c).to(BF16)
    q, s = pe.pe_rmsnorm_fp8(x, w)
    tq, ts = pe.pe_rmsnorm_fp8(x[-tail:].contiguous(), w)
    assert torch.equal(q[-tail:].float(), tq.float()) and torch.equal(s[:, -tail:], ts)
    del q, s
    first = n - n % 128 - 128                                  # tiles of 128 rows
    q, s, qt, st = pe.pe_quantize_fp8(x, transposed=True)
    tq, ts, tqt, tst = pe.pe_quantize_fp8(x[first:].contiguous(), transposed=True)
    assert torch.equal(q[first:].float(), tq.float()) and torch.equal(s[:, first:], ts)
    assert torch.equal(qt[:, first:].float(), tqt.float())
    assert torch.equal(st[first // 128:], tst)
    del qt, st
    wq, ws = pe.pe_quantize_fp8(_randn(492, 24, c), 128)
    out = pe.pe_matmul_fp8(q, s, wq, ws)
    assert torch.equal(out[-4000:], pe.pe_matmul_fp8(q[-4000:], s[:, -4000:].contiguous(), wq, ws))
    del q, s, out
    dx, _ = pe.pe_rmsnorm_bwd(x, x, w)
    tx = x[-tail:].contiguous()
    assert torch.equal(dx[-tail:], pe.pe_rmsnorm_bwd(tx, tx, w)[0])


def test_an_output_of_more_than_two_to_the_31_elements():
    m, n, k = 70001, 32768, 128
    a, sa = pe.pe_quantize_fp8(_randn(495, m, k))
    b, sb = pe.pe_quantize_fp8(_randn(496, n, k), 128)
    out = pe.pe_matmul_fp8(a, sa, b, sb)
    for rows in (slice(0, 300), slice(m - 300, m)):
        part = pe.pe_matmul_fp8(a[rows], sa[:, rows].contiguous(), b, sb)
        assert torch.equal(out[rows], part)
    odd = pe.pe_matmul_fp8(a, sa, b[:-1], sb)                  # rows that start anywhere
    assert torch.equal(odd[-300:], out[-300:, :-1])


def test_refused_tensors():
    x, w = torch.zeros(4, 64, device=DEV), torch.ones(64, device=DEV)
    q, s = pe.pe_quantize_fp8(x)
    wq, ws = pe.pe_quantize_fp8(torch.ones(8, 64, device=DEV), 128)
    half = torch.float16
    bad = [
        (ValueError, lambda: pe.pe_rmsnorm(x, torch.ones(63, device=DEV))),
        (ValueError, lambda: pe.pe_rmsnorm(x.view(2, 2, 64), w)),
        (ValueError, lambda: pe.pe_rmsnorm(x, w, residual=x[:3])),
        (ValueError, lambda: pe.pe_rmsnorm(x, w, residual=x.to(BF16))),
        (ValueError, lambda: pe.pe_rmsnorm(x, w, out=torch.empty(64, 4, device=DEV).t())),
        (ValueError, lambda: pe.pe_rmsnorm(x, w, residual_out=x)),
        (TypeError, lambda: pe.pe_rmsnorm(x.to(half), w)),
        (TypeError, lambda: pe.pe_rmsnorm_fp8(x, w, dtype=torch.int8)),
        (ValueError, lambda: pe.pe_rmsnorm_fp8(x, w, out=q[:3])),
        (ValueError, lambda: pe.pe_rmsnorm_fp8(x, w, dtype=E5M2, out=q)),
        (ValueError, lambda: pe.pe_rmsnorm_bwd(x, x[:3], w)),
        (ValueError, lambda: pe.pe_rmsnorm_bwd(x.to(BF16), x, w)),
        (ValueError, lambda: pe.pe_rmsnorm_bwd(x, x, w, dresidual=x[:, :63])),
        (ValueError, lambda: pe.pe_quantize_fp8(x, 64)),
        (ValueError, lambda: pe.pe_quantize_fp8(x, plain=False)),
        (ValueError, lambda: pe.pe_quantize_fp8(x[0])),
        (TypeError, lambda: pe.pe_quantize_fp8(x.to(half))),
        (ValueError, lambda: pe.pe_matmul_fp8(q, s[:, :3], wq, ws)),
        (ValueError, lambda: pe.pe_matmul_fp8(q, s, wq, ws.double())),
        (ValueError, lambda: pe.pe_matmul_fp8(q, s, wq[:, :48], ws)),
        (ValueError, lambda: pe.pe_matmul_fp8(q, s, wq, ws, out=torch.empty(4, 7, device=DEV))),
        (ValueError, lambda: pe.pe_matmul_fp8(q[0], s, wq, ws)),
        (TypeError, lambda: pe.pe_matmul_fp8(x, s, wq, ws)),
        (TypeError, lambda: pe.pe_matmul_fp8(q, s, wq, ws, dtype=half)),
        (ValueError, lambda: pe.pe_matmul_fp8(q.cpu(), s, wq, ws)),
        (ValueError, lambda: pe.pe_matmul_fp8(q, s.cpu(), wq, ws)),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()
    with pytest.raises(pe.PackedAttentionError) as e:
        pe.pe_rmsnorm(x, w, eps=0.0)
    assert e.value.status == 1
    wide = torch.zeros(2, 16385, device=DEV)
    with pytest.raises(pe.PackedAttentionError) as e:
        pe.pe_rmsnorm_bwd(wide, wide, wide[0])
    assert e.value.status == 4
