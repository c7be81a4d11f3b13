"""Sizes at the ends of the integer types: refused on the host, before any launch (the
addresses here are fake and never read)."""

import pytest

from test_fp8_host import OK, OVERFLOW, UNSUPPORTED, _bwd, _norm, _norm8, lib  # noqa: F401


@pytest.mark.parametrize("below", [1, 2, 128, 255, 256, 1024])
def test_norms_of_nearly_two_to_the_31_channels_are_refused(lib, below):  # noqa: F811
    """A warp's step past the last channel has to stay below 2^31."""
    c = (1 << 31) - below
    assert _norm(lib, c=c) == OVERFLOW
    assert _norm8(lib, c=c, ld=1 << 32) == OVERFLOW
    assert _bwd(lib, c=c) == UNSUPPORTED
    assert _norm(lib, c=c, n=0) == OVERFLOW
    assert _norm(lib, c=1 << 20, n=0) == OK
