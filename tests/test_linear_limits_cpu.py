"""Limits and refusals of the linear layer that need no GPU: sizes, alignment, workspaces."""
import ctypes

import pytest

moe = pytest.importorskip("combine_overlap_b200.moe")

HUGE = ctypes.c_size_t(-1).value
BIG = 2 ** 30


@pytest.mark.parametrize("shape,ok", [((BIG, 1, 1), True), ((BIG + 1, 1, 1), False), ((1, BIG + 1, 1), False),
                                      ((1, 1, BIG + 1), False), ((0, 4, 4), False), ((4, 0, 4), False), ((4, 4, 0), False),
                                      ((-1, 4, 4), False), ((2 ** 20, 2 ** 20, 1), False), ((2 ** 19, 2 ** 20, 1), True)])
def test_shapes(shape, ok):
    assert (moe._lib.moe_linear_workspace_size(*shape) != HUGE) == ok
    assert (moe._lib.moe_linear_backward_workspace_size(*shape) != HUGE) == ok


def _call(M=64, K=64, N=64, x=4096, W=8192, bias=0, residual=0, act=0, code=0, out=16384, pre=0, ws=None, n=0):
    return moe._lib.moe_linear(moe._LINEAR.pack(M, K, N, x, W, bias, residual, act, code, out, pre), ws, n, None)


def test_pointers_and_workspaces_are_checked_before_any_launch():
    for bad in (dict(x=0), dict(W=0), dict(out=0), dict(x=4098), dict(W=8200), dict(bias=4), dict(residual=2),
                dict(out=16392), dict(pre=8), dict(act=4), dict(act=-1), dict(code=2)):
        assert _call(**bad) == moe.MOE_ERR_INVALID, bad
    assert _call(M=BIG + 1) == moe.MOE_ERR_UNSUPPORTED
    # rows of 65 elements need padded copies, and those a workspace
    need = moe.linear_workspace_size(200, 65, 64)
    assert need >= 200 * 72 * 2
    assert _call(M=200, K=65) == moe.MOE_ERR_WORKSPACE
    assert _call(M=200, K=65, ws=4096, n=need - 1) == moe.MOE_ERR_WORKSPACE
    assert _call(M=200, K=65, ws=4104, n=need) == moe.MOE_ERR_WORKSPACE
    assert moe.linear_workspace_size(200, 64, 64) == 0 and moe.linear_workspace_size(1, 65, 63) == 0


def test_the_packed_arguments_are_the_structures():
    """The binding's packed bytes read back through the structures of the header."""
    a = moe.LinearArgs.from_buffer_copy(moe._LINEAR.pack(1, 2, 3, 16, 32, 48, 64, 2, 1, 80, 96))
    assert [getattr(a, f) for f, _ in a._fields_] == [1, 2, 3, 16, 32, 48, 64, 2, 1, 80, 96]
    b = moe.LinearBwdArgs.from_buffer_copy(moe._LINEAR_BWD.pack(1, 2, 3, 16, 32, 48, 64, 3, 1, 0, 80, 96, 112))
    assert [getattr(b, f) for f, _ in b._fields_] == [1, 2, 3, 16, 32, 48, 64, 3, 1, 0, 80, 96, 112]
    r = moe.RouterArgs.from_buffer_copy(moe._ROUTER.pack(1, 16, 8, 4, 1, 1, 2.5))
    assert [getattr(r, f) for f, _ in r._fields_] == [1, 16, 8, 4, 1, 1, 2.5]
