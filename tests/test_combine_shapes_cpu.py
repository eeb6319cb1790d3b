"""Which shapes moe_combine_rows and its gradient take: T, d, E and k count, the other fields do not.
With T = 0 nothing is launched, so no call here reaches a device."""
import ctypes

import pytest

from sparse_mixture_experts_17_b200 import build as B
from sparse_mixture_experts_17_b200 import moe as M


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.lib()


def _both(lib, s):
    a = lib.moe_combine_rows(ctypes.byref(s), None, None, None, None, None, None, None)
    b = lib.moe_combine_rows_backward(ctypes.byref(s), None, None, None, None, None, None, None, None)
    assert a == b
    return a


@pytest.mark.parametrize("d", [8, 24, 200, 1000, 32776, 65536])
def test_widths_that_a_linear_product_writes(lib, d):
    assert _both(lib, M.make_shape(0, d, 0, 8, 2)) == M.MOE_OK
    assert _both(lib, M.make_shape(0, d, -5, 8, 8, capacity=7, d_ff_shared=3)) == M.MOE_OK


@pytest.mark.parametrize("T,d,E,k", [(-1, 128, 8, 2), ((1 << 24) + 1, 128, 8, 2), (0, 0, 8, 2), (0, -8, 8, 2), (0, 4, 8, 2),
                                     (0, 100, 8, 2), (0, 65544, 8, 2), (0, 128, 0, 1), (0, 128, 257, 2), (0, 128, 8, 0),
                                     (0, 128, 8, 9), (0, 128, 32, 17)])
def test_refusals(lib, T, d, E, k):
    assert _both(lib, M.make_shape(T, d, 128, E, k)) == M.MOE_ERR_INVALID_ARG
