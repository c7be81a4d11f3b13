"""Tensors that do not start at a multiple of their elements' size are refused before any kernel
could read them."""

import ctypes

import pytest
import torch

from test_tail_bwd_host import GEGLU, NONE, UNSUPPORTED, WORKSPACE, _act, _ln, lib  # noqa: F401

DEV = "cuda:0"


# The calls lack a workspace that they need: what is refused for that is aligned.

@pytest.mark.parametrize("dtype,off", [(0, 1), (1, 1), (1, 2)])
def test_layernorm_bwd(lib, dtype, off):  # noqa: F811
    args = dict(dtype=dtype, n=9000, dr=16, ws=None)
    assert _ln(lib, **args) == WORKSPACE
    for name in ("dy", "h", "w", "dr", "dx"):
        assert _ln(lib, **{**args, name: 64 + off}) == UNSUPPORTED
    for name in ("dw", "db"):
        assert _ln(lib, **{**args, name: 66}) == UNSUPPORTED


@pytest.mark.parametrize("dtype,off", [(0, 1), (1, 1), (1, 2)])
def test_activation_bwd(lib, dtype, off):  # noqa: F811
    args = dict(dtype=dtype, act=GEGLU, n=9000, ws=None)
    assert _act(lib, **args) == WORKSPACE
    for name in ("dy", "z", "dz"):
        assert _act(lib, **{**args, name: 64 + off}) == UNSUPPORTED
    assert _act(lib, **{**args, "db": 66}) == UNSUPPORTED
    sums = dict(args, act=NONE, z=None, dz=None)
    assert _act(lib, **sums) == WORKSPACE
    assert _act(lib, **{**sums, "dy": 64 + off}) == UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,off", [(0, 1), (1, 1), (1, 2)])
def test_dropout_and_rotary_positions(lib, dtype, off):  # noqa: F811
    size = 4 if dtype else 2
    x, y, r = (torch.zeros(4096, dtype=torch.uint8, device=DEV) for _ in range(3))
    at = {"x": x.data_ptr(), "y": y.data_ptr(), "r": r.data_ptr()}

    def drop(**kw):
        a = {**at, **kw}
        return lib.pe_dropout(dtype, a["x"], a["r"], 100, 0.5, 1, 2, None, a["y"], None)

    assert drop() == 0
    for name, p in at.items():
        assert drop(**{name: p + off}) == UNSUPPORTED
        assert drop(**{name: p + size}) == 0
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    sections = (ctypes.c_int32 * 1)(16)
    at = {"q": x.data_ptr(), "qo": y.data_ptr(), "k": r.data_ptr(), "ko": r.data_ptr(),
          "pos": pos.data_ptr()}

    def rope(heads=1, **kw):
        a = {**at, **kw}
        return lib.pe_rope_axes(dtype, a["q"], 32, a["qo"], 32, 1, a["k"], 32, a["ko"], 32, heads,
                                a["pos"], sections, 1, 3, 32, 1e4, 0, 0, None)

    assert rope() == 0
    for name, p in at.items():
        assert rope(**{name: p + off}) == UNSUPPORTED
    assert rope(heads=0, k=at["k"] + off, ko=at["ko"] + off) == 0      # not read
    assert rope(q=at["q"] + size, k=None, ko=None, heads=0) == 0
    torch.cuda.synchronize()
