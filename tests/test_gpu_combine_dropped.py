"""The combine's gradient where slots are dropped and the caller brings no dy."""
import pytest
import torch

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")


@pytest.mark.parametrize("T,d,k", [(1, 64, 2), (200, 512, 6)])
def test_rows_without_a_slot_are_zero_in_a_dy_made_here(T, d, k):
    g = torch.Generator(device="cuda").manual_seed(T)
    dout, y = (torch.randn(n, d, generator=g, device="cuda").bfloat16() for n in (T, T * k))
    gate = torch.rand(T, k, generator=g, device="cuda") + 0.5
    row_of = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    row_of[1::3] = -1
    torch.full((T * k, d), float("nan"), dtype=torch.bfloat16, device="cuda")    # what the allocator hands out again
    dy, _ = moe.combine_backward(dout, y, row_of, gate)
    named = torch.zeros(T * k, dtype=torch.bool, device="cuda")
    named[row_of[row_of >= 0].long()] = True
    assert not dy[~named].any() and dy[named].any(1).all()
    mine = torch.full((T * k, d), 3.0, dtype=torch.bfloat16, device="cuda")
    moe.combine_backward(dout, y, row_of, gate, dy=mine)
    assert (mine[~named] == 3).all() and torch.equal(mine[named], dy[named])
