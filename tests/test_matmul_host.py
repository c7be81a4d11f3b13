"""Host-side checks of the 16- and 32-bit matrix product: every refusal answers without a GPU
and launches nothing (the addresses here are fake and never read)."""

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
NONE, RELU, GELU, GEGLU = 0, 1, 2, 3


def _mm(lib, **kw):
    a = dict(dtype=0, a=16, lda=64, ta=0, b=32, ldb=64, tb=0, m=4, n=8, k=64, bias=None, act=NONE,
             res=None, ldr=8, out_dtype=0, out=48, ldo=8, pre=None, ldp=8, ws=16, size=1 << 44)
    a.update(kw)
    return lib.pe_matmul(a["dtype"], a["a"], a["lda"], a["ta"], a["b"], a["ldb"], a["tb"], a["m"],
                         a["n"], a["k"], a["bias"], a["act"], a["res"], a["ldr"], a["out_dtype"],
                         a["out"], a["ldo"], a["pre"], a["ldp"], a["ws"], a["size"], None)


def test_types_and_activations(lib):
    assert _mm(lib, dtype=2) == UNSUPPORTED
    assert _mm(lib, out_dtype=-1) == UNSUPPORTED
    assert _mm(lib, act=4) == INVALID
    assert _mm(lib, act=-1) == INVALID
    assert _mm(lib, act=GEGLU, n=7, ldo=8) == INVALID


def test_sizes(lib):
    for name in ("m", "n", "k"):
        assert _mm(lib, **{name: -1}) == INVALID
    big = (1 << 31) - 1024
    assert _mm(lib, m=big) == OVERFLOW
    assert _mm(lib, n=big, ldo=big) == OVERFLOW
    assert _mm(lib, k=big // 6, lda=big, ldb=big) == OVERFLOW
    assert _mm(lib, m=1 << 30, n=1 << 30, ldo=1 << 30) == OVERFLOW
    assert _mm(lib, m=1 << 30, n=1 << 30, ldo=1 << 30, k=0) == OVERFLOW
    assert _mm(lib, m=0, a=None, out=None) == OK
    assert _mm(lib, n=0, b=None, out=None) == OK


def test_pointers_and_strides(lib):
    for name in ("a", "b", "out"):
        assert _mm(lib, **{name: None}) == INVALID
    assert _mm(lib, lda=56) == INVALID
    assert _mm(lib, ldb=56) == INVALID
    assert _mm(lib, ldo=7) == INVALID
    assert _mm(lib, res=16, ldr=7) == INVALID
    assert _mm(lib, pre=64, ldp=7) == INVALID
    assert _mm(lib, ta=1, m=72, lda=64) == INVALID
    assert _mm(lib, tb=1, n=72, ldb=64, ldo=72) == INVALID
    assert _mm(lib, pre=48) == INVALID                         # out itself
    assert _mm(lib, pre=16, res=16) == INVALID
    assert _mm(lib, out=48, res=48, ldr=16) == INVALID         # two strides of one buffer
    for name in ("lda", "ldb", "ldo"):
        assert _mm(lib, **{name: 1 << 37}) == OVERFLOW
    assert _mm(lib, a=24) == UNSUPPORTED
    assert _mm(lib, b=8) == UNSUPPORTED
    assert _mm(lib, lda=68) == UNSUPPORTED
    assert _mm(lib, ldb=65) == UNSUPPORTED
    assert _mm(lib, dtype=1, a=18) == UNSUPPORTED
    assert _mm(lib, out=49) == UNSUPPORTED
    assert _mm(lib, bias=17) == UNSUPPORTED
    assert _mm(lib, out_dtype=1, out=50) == UNSUPPORTED
    # The up part's columns of a transposed b would not start at a multiple of 16 bytes.
    assert _mm(lib, act=GEGLU, tb=1, n=24, ldb=24, ldo=12) == UNSUPPORTED


def test_workspace(lib):
    size = lib.pe_matmul_workspace_size
    assert size(0, 0, 0, 169151, 1024, 1024, NONE) == 0
    assert size(0, 1, 1, 2304, 768, 32299, NONE) > 0           # runs of blocks
    assert size(2, 0, 0, 4, 8, 64, NONE) == 0
    assert size(0, 0, 0, 4, 8, 64, 9) == 0
    assert size(0, 0, 0, 4, -8, 64, NONE) == 0
    # Three parts of two bytes an element, rows rounded up to eight elements.
    assert size(1, 0, 1, 5, 7, 9, NONE) == 6 * (5 * 16 + 9 * 8)
    assert size(1, 1, 0, 5, 7, 9, NONE) == 6 * (9 * 8 + 7 * 16)
    need = size(1, 0, 1, 4, 8, 64, NONE)
    assert _mm(lib, dtype=1, tb=1, size=need - 1) == WORKSPACE
    assert _mm(lib, dtype=1, tb=1, ws=None) == WORKSPACE
    assert _mm(lib, dtype=1, tb=1, ws=24) == WORKSPACE
    # Few products, neither operand transposed: multiplied as they lie.
    assert size(1, 0, 0, 4, 100000, 4096, NONE) == 0
    assert size(1, 0, 0, 64, 100, 1000, NONE) == 0
    assert size(1, 0, 0, 320, 1000, 1000, NONE) == 6 * (320 + 1000) * 1000


def test_binding_refuses_before_any_call(lib):
    import padding_free_packed_gb300 as pe
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        pe.pe_matmul(x, x)
    with pytest.raises(ValueError, match="activation"):
        pe.pe_matmul(x, x, activation="silu")
