"""Host-side checks of the layer tail's backward calls, dropout and rotary positions with
several axes: every refusal answers without a GPU and launches nothing (the addresses here
are fake and never read)."""

import ctypes

import pytest
import torch

import tail_reference as ref


@pytest.fixture(scope="module")
def lib():
    from padding_free_packed_gb300 import binding
    from padding_free_packed_gb300 import build
    if build.is_stale():
        build.build()
    return binding.load_library()


OK, INVALID, OVERFLOW, UNSUPPORTED, WORKSPACE = 0, 1, 3, 4, 5
NONE, RELU, GELU, GEGLU = 0, 1, 2, 3


def _ln(lib, **kw):
    a = dict(dtype=0, dy=16, h=16, w=16, dr=None, n=4, c=64, eps=1e-5, dx=16, dw=16, db=16, ws=16,
             size=1 << 30)
    a.update(kw)
    return lib.pe_layernorm_bwd(a["dtype"], a["dy"], a["h"], a["w"], a["dr"], a["n"], a["c"],
                                a["eps"], a["dx"], a["dw"], a["db"], a["ws"], a["size"], None)


def _act(lib, **kw):
    a = dict(dtype=0, act=GELU, dy=16, z=32, n=4, f=64, dz=48, db=16, ws=16, size=1 << 40)
    a.update(kw)
    return lib.pe_activation_bwd(a["dtype"], a["act"], a["dy"], a["z"], a["n"], a["f"], a["dz"],
                                 a["db"], a["ws"], a["size"], None)


def _drop(lib, **kw):
    a = dict(dtype=0, x=16, r=None, n=4, p=0.5, seed=1, offset=2, dev=None, y=16)
    a.update(kw)
    return lib.pe_dropout(a["dtype"], a["x"], a["r"], a["n"], a["p"], a["seed"], a["offset"],
                          a["dev"], a["y"], None)


def _rope(lib, **kw):
    a = dict(dtype=0, q=16, qs=128, qo=16, qos=128, qh=2, k=32, ks=64, ko=32, kos=64, kh=1, pos=16,
             sections=(16, 16), axes=None, n=4, d=64, theta=1e4)
    a.update(kw)
    s = a["sections"]
    cs = None if s is None else (ctypes.c_int32 * max(len(s), 1))(*s)
    axes = a["axes"] if a["axes"] is not None else len(s)
    return lib.pe_rope_axes(a["dtype"], a["q"], a["qs"], a["qo"], a["qos"], a["qh"], a["k"],
                            a["ks"], a["ko"], a["kos"], a["kh"], a["pos"], cs, axes, a["n"],
                            a["d"], a["theta"], 0, 0, None)


def test_layernorm_bwd_refusals(lib):
    assert _ln(lib, dtype=2) == UNSUPPORTED
    assert _ln(lib, n=-1) == INVALID
    assert _ln(lib, c=0) == INVALID
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert _ln(lib, eps=eps) == INVALID
    for name in ("dy", "h", "w", "dx", "dw"):
        assert _ln(lib, **{name: None}) == INVALID
    assert _ln(lib, c=16385) == UNSUPPORTED
    need = lib.pe_layernorm_bwd_workspace_size(5000, 64)
    assert need > 0
    assert _ln(lib, n=5000, size=need - 1) == WORKSPACE
    assert _ln(lib, n=5000, ws=None) == WORKSPACE
    assert _ln(lib, n=5000, ws=24) == WORKSPACE
    assert lib.pe_layernorm_bwd_workspace_size(4, 64) == 0     # few rows need none
    assert lib.pe_layernorm_bwd_workspace_size(1, 5000) > 0
    assert lib.pe_layernorm_bwd_workspace_size(0, 64) == 0
    assert lib.pe_layernorm_bwd_workspace_size(5000, 0) == 0
    assert lib.pe_layernorm_bwd_workspace_size(5000, 16385) == 0


def test_activation_bwd_refusals(lib):
    assert _act(lib, dtype=2) == UNSUPPORTED
    assert _act(lib, act=4) == INVALID
    assert _act(lib, act=-1) == INVALID
    assert _act(lib, n=-1) == INVALID
    assert _act(lib, f=0) == INVALID
    assert _act(lib, f=(1 << 30)) == OVERFLOW
    for name in ("dy", "z", "dz"):
        assert _act(lib, **{name: None}) == INVALID
    assert _act(lib, act=GEGLU, dz=16) == INVALID              # dz = dy is half as wide
    assert _act(lib, act=NONE, z=None) == INVALID              # dz is dy itself
    assert _act(lib, act=NONE, dz=None) == INVALID
    assert _act(lib, act=NONE, z=None, dz=None, db=None) == INVALID
    for act, wide in ((GELU, 1), (GEGLU, 2)):
        need = lib.pe_activation_bwd_workspace_size(act, 9000, 64)
        assert need == wide * lib.pe_activation_bwd_workspace_size(RELU, 9000, 64) > 0
        assert _act(lib, act=act, n=9000, size=need - 1) == WORKSPACE
    assert _act(lib, n=9000, ws=None) == WORKSPACE
    assert lib.pe_activation_bwd_workspace_size(GELU, 4, 64) == 0      # few rows need none
    assert lib.pe_activation_bwd_workspace_size(7, 9000, 64) == 0
    assert lib.pe_activation_bwd_workspace_size(GELU, 9000, 0) == 0


def test_dropout_refusals(lib):
    assert _drop(lib, dtype=2) == UNSUPPORTED
    assert _drop(lib, n=-1) == INVALID
    for p in (-0.1, 1.0, 2.0, float("nan")):
        assert _drop(lib, p=p) == INVALID
    assert _drop(lib, x=None) == INVALID
    assert _drop(lib, y=None) == INVALID
    assert _drop(lib, n=(1 << 60) + 1) == OVERFLOW
    assert _drop(lib, dev=20) == UNSUPPORTED
    assert _drop(lib, n=0, x=None, y=None) == OK


def test_rope_axes_refusals(lib):
    assert _rope(lib, dtype=2) == UNSUPPORTED
    for bad in (dict(n=-1), dict(qh=-1), dict(kh=-1), dict(d=63), dict(d=0), dict(d=258),
                dict(theta=1.0), dict(theta=float("nan")), dict(theta=float("inf")),
                dict(sections=None, axes=1), dict(sections=(16, 15)), dict(sections=(16, 17)),
                dict(sections=(33, -1)), dict(sections=(), axes=0),
                dict(sections=(8, 8, 8, 4, 4)), dict(pos=None), dict(q=None), dict(qo=None),
                dict(k=None), dict(ko=None), dict(qs=127, qos=127), dict(kos=60),
                dict(qs=256)):                                 # in place with two strides
        assert _rope(lib, **bad) == INVALID, bad
    assert _rope(lib, qh=1 << 23) == OVERFLOW
    assert _rope(lib, n=0) == OK
    assert _rope(lib, qh=0, kh=0) == OK


def test_bindings_refuse_before_any_call(lib):
    import padding_free_packed_gb300 as pe
    x = torch.zeros(4, 8)
    for call in (lambda: pe.pe_layernorm_bwd(x, x, x[0]), lambda: pe.pe_dropout(x, 0.5, 1),
                 lambda: pe.pe_activation_bwd(x, x, "gelu"),
                 lambda: pe.pe_rope_axes(x.view(4, 1, 8), None, torch.zeros(1, 4).int(), (4,),
                                         1e4)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="activation"):
        pe.pe_activation_bwd(x, x, "tanh")


def test_reference_draws_the_published_numbers():
    """Philox4x32-10's known answers of its authors' distribution."""
    assert [hex(w) for w in ref.philox_words(0, 0, 0)] == [
        "0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    ones = 2 ** 64 - 1
    assert [hex(w) for w in ref.philox_words(ones, ones, ones)] == [
        "0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]
    # counter 243f6a88 85a308d3 13198a2e 03707344, key a4093822 299f31d0
    assert [hex(w) for w in ref.philox_words(0x85a308d3243f6a88, 0x299f31d0a4093822,
                                             0x0370734413198a2e)] == [
        "0xd16cfe09", "0x94fdcceb", "0x5001e420", "0x24126ea1"]
