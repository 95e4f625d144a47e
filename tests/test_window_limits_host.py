"""Calls of windowed attention that are too long to be planned are refused on the host as sizes, not
as a failed launch."""
import ctypes

import pytest

import int4_group_quantized_gs64_gb300 as q

ESHAPE = -2
P = ctypes.c_void_p(0x10000)  # aligned and never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    q.build()
    return q.lib()


@pytest.mark.parametrize("T,G,W", [(1 << 22, 8, 2 ** 31 - 1), (1 << 22, 128, 1 << 28), (1 << 19, 64, 1 << 30)])
def test_too_many_steps(L, T, G, W):
    d = q.AttnCacheDesc(0x10000, 0x10000, 8, 8, 256, 64, 1)
    assert L.attn_window(ctypes.byref(d), P, 8 * G * 64, 8 * G, P, 1 << 22, P, P, 1, T, T, W, 0, 0.1, P, 1, P, None, P,
                         1 << 50, None) == ESHAPE
