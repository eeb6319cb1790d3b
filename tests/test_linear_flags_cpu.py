"""moe_linear_t.flags: the test-only timeout flag alone is taken."""
import ctypes

import pytest

from sparse_mixture_experts_17_b200 import build as B
from sparse_mixture_experts_17_b200 import moe as M


@pytest.fixture(scope="module")
def lib():
    B.build()
    return M.lib()


@pytest.mark.parametrize("bit", range(32))
def test_flags(lib, bit):
    flags = ctypes.c_int32(1 << bit).value
    want = M.MOE_OK if flags == M.MOE_FLAG_TEST_TIMEOUT else M.MOE_ERR_INVALID_ARG
    s, n = M.make_linear(64, 128, 256, flags=flags), ctypes.c_size_t(0)
    assert lib.moe_linear_workspace_size(ctypes.byref(s), ctypes.byref(n)) == want
    none = M.make_linear(0, 128, 256, flags=flags)       # no rows: nothing is launched
    assert lib.moe_linear_forward(ctypes.byref(none), *[None] * 9) == want
    assert lib.moe_linear_backward(ctypes.byref(none), *[None] * 10, 0, None) == want
