"""Failure detection in the linear layer without a GPU fault: the debug setting withholds the
first tile's operands, so that the waits for them run out after their bound; the kernel counts
that and returns, and the next call is right."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")

BF, F32 = torch.bfloat16, torch.float32
LIMIT_US = 20000


def _rand(seed, *shape, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# a block, a pair, blocks and pairs whose reduction is split over a cluster, several tiles to a block
@pytest.mark.parametrize("cg,bn,s,M", [(1, 128, 1, 300), (2, 256, 1, 300), (1, 128, 4, 300), (2, 128, 2, 300), (1, 32, 1, 9000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_withheld_operand_is_a_timeout_and_the_next_call_is_right(cg, bn, s, M, dtype):
    x, W = _rand(1, M, 2048), _rand(2, 2048, 520)
    with moe.linear_debug(cg, bn, s):
        want = moe.linear(x, W, out_dtype=dtype)
        assert moe.linear_get_status() == moe.MOE_OK
        before = moe.linear_timeouts()
        with moe.linear_debug(cg, bn, s, timeout_us=LIMIT_US, withhold=True):
            moe.linear(x, W, out_dtype=dtype)
        assert moe.linear_get_status() == moe.MOE_ERR_TIMEOUT
        assert moe.linear_timeouts() > before
        assert moe.linear_get_status() == moe.MOE_OK
    with moe.linear_debug(cg, bn, s):
        assert torch.equal(moe.linear(x, W, out_dtype=dtype), want)
    assert moe.linear_get_status() == moe.MOE_OK


@pytest.mark.parametrize("cg,sw", [(1, 4), (2, 3)])
def test_a_withheld_operand_of_slices(cg, sw):
    x, W, dout = _rand(1, 4096, 264), _rand(2, 264, 128), _rand(3, 4096, 128, dtype=F32)
    f = lambda: moe.linear_backward(dout, x, W, want_dx=False)[1]  # noqa: E731
    with moe.linear_debug(cg, 64, 1, sw):
        want = f()
    with moe.linear_debug(cg, 64, 1, sw, timeout_us=LIMIT_US, withhold=True):
        f()
    assert moe.linear_get_status() == moe.MOE_ERR_TIMEOUT
    with moe.linear_debug(cg, 64, 1, sw):
        assert torch.equal(f(), want)
    assert moe.linear_get_status() == moe.MOE_OK


def test_one_thread_does_not_clear_what_another_has_not_seen():
    x, W = _rand(1, 300, 512), _rand(2, 512, 520)
    assert moe.linear_get_status() in (moe.MOE_OK, moe.MOE_ERR_TIMEOUT)   # what came before
    seen = []

    def other(go, done):
        seen.append(moe.linear_get_status())              # whatever there was before
        done.set()
        go.wait()
        seen.append(moe.linear_get_status())
        seen.append(moe.linear_get_status())

    go, done = threading.Event(), threading.Event()
    t = threading.Thread(target=other, args=(go, done))
    t.start()
    done.wait()
    with moe.linear_debug(timeout_us=LIMIT_US, withhold=True):
        moe.linear(x, W)
    assert moe.linear_get_status() == moe.MOE_ERR_TIMEOUT and moe.linear_get_status() == moe.MOE_OK
    go.set()
    t.join()
    assert seen[1:] == [moe.MOE_ERR_TIMEOUT, moe.MOE_OK]


def test_settings_are_the_threads_own():
    """A setting of one thread changes no other thread's products."""
    x, W = _rand(1, 300, 512), _rand(2, 512, 520)
    assert moe.linear_get_status() in (moe.MOE_OK, moe.MOE_ERR_TIMEOUT)
    want, got = moe.linear(x, W), []
    with moe.linear_debug(cg=1, bn=32, withhold=True, timeout_us=LIMIT_US):
        t = threading.Thread(target=lambda: got.append(moe.linear(x, W)))
        t.start()
        t.join()
    assert torch.equal(got[0], want) and moe.linear_get_status() == moe.MOE_OK
