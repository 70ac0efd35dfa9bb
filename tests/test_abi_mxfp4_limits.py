"""Sizes that the MXFP4 product refuses on the host, before any HIP call (CPU only)."""

import ctypes

import pytest

from helpers import ensure_built

EUNSUP = 2
FAKE = ctypes.c_void_p(0x10000)        # aligned, never dereferenced: calls fail first


@pytest.fixture(scope="module")
def L():
    ensure_built()
    from precision_moe_numerics_nvfp4_amd import binding
    return binding.lib()


def test_product_tile_bounds(L):
    def f(rows, cap, N, K, G=1, tok=FAKE):
        return L.moe_fwd_grouped_gemm_mxfp4(FAKE, FAKE, rows, tok, FAKE, FAKE, FAKE, G, cap, N, K, FAKE, 1, None)
    # gathered from 2 GiB of codes: a workgroup to each 32 x 128
    assert f(1 << 20, 1 << 20, 32768, 4096) == EUNSUP
    assert f(1 << 30, 32, 1 << 28, 128, G=4000) == EUNSUP
    # else the count of 256 x 256 tiles stays an int
    assert f(64, (1 << 31) - 1, 65536, 128) == EUNSUP
    assert f((1 << 31) - 1, (1 << 31) - 1, 65536, 128, tok=None) == EUNSUP
    assert f(64, 64, 1 << 39, 128) == EUNSUP
