"""The linear layer's debug settings and its count of timeouts: what is refused before any CUDA call."""
import ctypes

import pytest

moe = pytest.importorskip("combine_overlap_b200.moe")


def _set(*args):
    return moe._lib.moe_linear_debug_set(ctypes.byref(moe.LinearDebug(*args)))


def test_settings():
    for bad in ((-1,), (1, 0, 1, 1), (1, 64, 0, 1), (2, 64, 1, 0), (1, -32, 1, 1), (0, 0, 0, 0, -5)):
        assert _set(*bad) == moe.MOE_ERR_INVALID, bad
    for good in ((), (0, 0, 0, 0, 20000, 1), (1, 64, 1, 1), (2, 256, 4, 1)):
        assert _set(*good) == moe.MOE_OK, good
    assert moe._lib.moe_linear_debug_set(None) == moe.MOE_OK
    assert moe._lib.moe_linear_timeouts(None, None) == moe.MOE_ERR_INVALID


def test_settings_nest_and_come_back():
    with moe.linear_debug(cg=1, bn=64):
        outer = moe._thread.linear_debug
        with moe.linear_debug(timeout_us=1000):
            assert moe._thread.linear_debug.timeout_us == 1000
        assert moe._thread.linear_debug is outer
        with pytest.raises(moe.MoEError):
            with moe.linear_debug(cg=-1):
                pass
        assert moe._thread.linear_debug is outer
    assert moe._thread.linear_debug is None
