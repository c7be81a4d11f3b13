"""Sizes at the ends of the integer types: refused on the host, before any launch (the
addresses here are fake and never read)."""

import pytest

from test_fp8_host import (INVALID, OK, OVERFLOW, UNSUPPORTED, _bwd, _mm, _norm,  # noqa: F401
                           _norm8, lib)


@pytest.mark.parametrize("below", [1, 2, 128, 255, 256, 1024])
def test_norms_of_nearly_two_to_the_31_channels_are_refused(lib, below):  # noqa: F811
    """A warp's step past the last channel has to stay below 2^31."""
    c = (1 << 31) - below
    assert _norm(lib, c=c) == OVERFLOW
    assert _norm8(lib, c=c, ld=1 << 32) == OVERFLOW
    assert _bwd(lib, c=c) == UNSUPPORTED
    assert _norm(lib, c=c, n=0) == OVERFLOW
    assert _norm(lib, c=1 << 20, n=0) == OK


@pytest.mark.parametrize("m,n,k", [((1 << 31) - 1100,) * 3, (1 << 23, 1 << 23, 1 << 7),
                                   (1 << 30, 1 << 30, 1 << 31 - 4), (1 << 20, 1 << 20, 1 << 20)])
def test_products_of_too_many_blocks_are_refused(lib, m, n, k):  # noqa: F811
    """2^30 blocks of 256 x 256 x 128 or more, also where their number passes 2^64."""
    assert _mm(lib, m=m, n=n, k=k, lda=1 << 32, ldb=1 << 32) == OVERFLOW
    assert lib.pe_matmul_fp8_workspace_size(m, n, k) == 0


def test_workspace_of_sizes_that_no_product_takes(lib):  # noqa: F811
    for size in (1 << 31, 1 << 40, (1 << 63) - 1):
        for sizes in ((size, 64, 64), (64, size, 64), (64, 64, size), (size, size, size)):
            assert lib.pe_matmul_fp8_workspace_size(*sizes) == 0
    assert lib.pe_matmul_fp8_workspace_size(2304, 768, 32299) > 0


# Beyond two 256 x 256 tiles for each of the 76 pairs of SMs, whole tiles in turn were
# faster wherever both ways were measured; only runs need a workspace.
@pytest.mark.parametrize("m,n,k,runs", [
    (8192, 8192, 8192, False), (12288, 12288, 8192, False), (5120, 5120, 5120, False),
    (4096, 4096, 16384, False), (20000, 512, 4096, False), (2304, 2304, 4096, False),
    (2304, 768, 4097, False), (2304, 1152, 9000, False), (2304, 768, 6000, True),
    (2304, 768, 32299, True), (2304, 2304, 8192, True), (2500, 999, 9001, True)])
def test_runs_of_blocks_are_for_few_tiles_with_long_sums(lib, m, n, k, runs):  # noqa: F811
    assert (lib.pe_matmul_fp8_workspace_size(m, n, k) > 0) == runs


def test_a_norm_and_its_sum_need_a_buffer_each(lib):  # noqa: F811
    assert _norm(lib, res=32, y=64, res_out=64) == INVALID
    assert _norm8(lib, res=32, y=64, res_out=64) == INVALID
    assert _norm(lib, res=32, y=64, res_out=64, n=0) == OK
