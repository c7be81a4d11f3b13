"""Host-side checks of the 8-bit layer calls: every refusal answers without a
GPU and launches nothing (the addresses here are fake and never read)."""

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from padding_free_packed_gb300 import binding
    from padding_free_packed_gb300 import build
    if build.is_stale():
        build.build()
    return binding.load_library()


OK, INVALID, OVERFLOW, UNSUPPORTED, WORKSPACE = 0, 1, 3, 4, 5


def _norm(lib, **kw):
    a = dict(dtype=0, x=16, res=None, w=16, n=4, c=64, eps=1e-5, y=16, res_out=None)
    a.update(kw)
    return lib.pe_rmsnorm(a["dtype"], a["x"], a["res"], a["w"], a["n"], a["c"], a["eps"], a["y"],
                          a["res_out"], None)


def _norm8(lib, **kw):
    a = dict(dtype=0, fp8=0, x=16, res=None, w=16, n=4, c=64, eps=1e-5, q=16, ld=64, s=16, y=None,
             res_out=None)
    a.update(kw)
    return lib.pe_rmsnorm_fp8(a["dtype"], a["fp8"], a["x"], a["res"], a["w"], a["n"], a["c"],
                              a["eps"], a["q"], a["ld"], a["s"], a["y"], a["res_out"], None)


def _bwd(lib, **kw):
    a = dict(dtype=0, dy=16, h=16, w=16, dr=None, n=4, c=64, eps=1e-5, dx=16, dw=16, ws=16,
             size=1 << 30)
    a.update(kw)
    return lib.pe_rmsnorm_bwd(a["dtype"], a["dy"], a["h"], a["w"], a["dr"], a["n"], a["c"],
                              a["eps"], a["dx"], a["dw"], a["ws"], a["size"], None)


def _quant(lib, **kw):
    a = dict(dtype=0, fp8=0, x=16, r=4, c=64, block=1, q=16, ld=64, s=16, qt=16, ldt=16, st=16)
    a.update(kw)
    return lib.pe_quantize_fp8(a["dtype"], a["fp8"], a["x"], a["r"], a["c"], a["block"], a["q"],
                               a["ld"], a["s"], a["qt"], a["ldt"], a["st"], None)


def _mm(lib, **kw):
    a = dict(ta=0, a=16, lda=64, sa=16, tb=0, b=16, ldb=64, sb=16, m=4, n=8, k=64, dtype=0, out=16,
             ws=16, size=1 << 40)
    a.update(kw)
    return lib.pe_matmul_fp8(a["ta"], a["a"], a["lda"], a["sa"], a["tb"], a["b"], a["ldb"],
                             a["sb"], a["m"], a["n"], a["k"], a["dtype"], a["out"], a["ws"],
                             a["size"], None)


@pytest.mark.parametrize("call", [_norm, _norm8])
def test_rmsnorm_refusals(lib, call):
    assert call(lib, dtype=2) == UNSUPPORTED
    assert call(lib, n=-1) == INVALID
    assert call(lib, c=0) == INVALID
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert call(lib, eps=eps) == INVALID
    assert call(lib, x=None) == INVALID
    assert call(lib, w=None) == INVALID
    assert call(lib, res_out=16) == INVALID          # without a residual
    assert call(lib, n=0, x=None, w=None) == OK      # nothing to do


def test_rmsnorm_output_refusals(lib):
    assert _norm(lib, y=None) == INVALID
    assert _norm8(lib, fp8=2) == UNSUPPORTED
    assert _norm8(lib, q=None) == INVALID
    assert _norm8(lib, s=None) == INVALID
    assert _norm8(lib, q=24) == UNSUPPORTED          # address
    assert _norm8(lib, ld=72) == UNSUPPORTED         # not a multiple of 16
    assert _norm8(lib, ld=48) == UNSUPPORTED         # shorter than a row


def test_rmsnorm_bwd_refusals(lib):
    assert lib.pe_rmsnorm_bwd_workspace_size(768) >= 4 * 768
    assert lib.pe_rmsnorm_bwd_workspace_size(0) == 0
    assert _bwd(lib, dtype=2) == UNSUPPORTED
    assert _bwd(lib, n=-1) == INVALID
    assert _bwd(lib, c=0) == INVALID
    assert _bwd(lib, c=16385) == UNSUPPORTED
    assert _bwd(lib, eps=0.0) == INVALID
    for name in ("dy", "h", "w", "dx", "dw"):
        assert _bwd(lib, **{name: None}) == INVALID
    assert _bwd(lib, ws=None) == WORKSPACE
    assert _bwd(lib, ws=24) == WORKSPACE
    assert _bwd(lib, size=lib.pe_rmsnorm_bwd_workspace_size(64) - 1) == WORKSPACE


def test_quantize_refusals(lib):
    assert _quant(lib, dtype=2) == UNSUPPORTED
    assert _quant(lib, fp8=-1) == UNSUPPORTED
    assert _quant(lib, r=-1) == INVALID
    assert _quant(lib, c=-1) == INVALID
    for block in (0, 2, 64, 256):
        assert _quant(lib, block=block) == INVALID
    assert _quant(lib, x=None) == INVALID
    assert _quant(lib, q=None, qt=None) == INVALID
    assert _quant(lib, s=None) == INVALID
    assert _quant(lib, st=None) == INVALID
    assert _quant(lib, q=8) == UNSUPPORTED
    assert _quant(lib, ld=63) == UNSUPPORTED
    assert _quant(lib, ldt=0) == UNSUPPORTED
    assert _quant(lib, r=1 << 31, ldt=1 << 31) == OVERFLOW
    assert _quant(lib, c=1 << 31, ld=1 << 31) == OVERFLOW
    assert _quant(lib, r=0) == OK
    assert _quant(lib, c=0) == OK


def test_matmul_refusals(lib):
    assert _mm(lib, ta=2) == UNSUPPORTED
    assert _mm(lib, tb=-1) == UNSUPPORTED
    assert _mm(lib, dtype=2) == UNSUPPORTED
    for name in ("m", "n", "k"):
        assert _mm(lib, **{name: -1}) == INVALID
        assert _mm(lib, **{name: 1 << 31, "lda": 1 << 31, "ldb": 1 << 31}) == OVERFLOW
    for name in ("a", "b", "sa", "sb", "out"):
        assert _mm(lib, **{name: None}) == INVALID
    assert _mm(lib, a=8) == UNSUPPORTED
    assert _mm(lib, b=24) == UNSUPPORTED
    assert _mm(lib, lda=72) == UNSUPPORTED
    assert _mm(lib, ldb=48) == UNSUPPORTED
    assert _mm(lib, m=0, out=None) == OK
    assert _mm(lib, n=0, out=None) == OK


def test_without_a_gpu_the_calls_are_unsupported(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _norm(lib) == _norm8(lib) == _bwd(lib) == _quant(lib) == _mm(lib) == UNSUPPORTED


def test_bindings_refuse_host_tensors_and_wrong_types():
    import padding_free_packed_gb300 as pe
    x, w = torch.zeros(4, 64), torch.ones(64)
    q = torch.zeros(4, 64).to(torch.float8_e4m3fn)
    s = torch.ones(1, 4)
    for call in (lambda: pe.pe_rmsnorm(x, w), lambda: pe.pe_rmsnorm_fp8(x, w),
                 lambda: pe.pe_rmsnorm_bwd(x, x, w), lambda: pe.pe_quantize_fp8(x),
                 lambda: pe.pe_matmul_fp8(q, s, q, s)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
