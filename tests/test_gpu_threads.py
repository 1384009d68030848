"""Each entry point as the first CUDA call of a thread of its own, which no call has bound to the
device's context yet."""
import threading

import pytest
import torch

from combine_overlap_b200 import synth

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")

BF, F32 = torch.bfloat16, torch.float32


def _same_in_a_new_thread(f):
    want, got = f(), []
    torch.cuda.synchronize()

    def run():
        try:
            got.append(f())
            torch.cuda.synchronize()
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if isinstance(got[0], Exception):
        raise got[0]
    for a, b in zip(want, got[0]):
        assert torch.equal(a, b)


def _rand(seed, *shape, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("M,K,N", [(1, 256, 60), (300, 512, 520), (300, 65, 67)])
def test_linear(M, K, N):
    x, W = _rand(1, M, K), _rand(2, K, N)
    ws = torch.empty(max(1, moe.linear_workspace_size(M, K, N)), dtype=torch.uint8, device="cuda")
    out = torch.empty(M, N, dtype=BF, device="cuda")
    _same_in_a_new_thread(lambda: (moe.linear(x, W, out=out, ws=ws).clone(),))
    _same_in_a_new_thread(lambda: (moe.linear(x, W),))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_backward(dtype):
    x, W, dout = _rand(1, 300, 512), _rand(2, 512, 520), _rand(3, 300, 520, dtype=dtype)
    _same_in_a_new_thread(lambda: moe.linear_backward(dout, x, W)[:2])


def test_router():
    z, dg = _rand(1, 100, 64, dtype=F32), _rand(2, 100, 6, dtype=F32)
    idx = moe.route_scored(z, 6)[0]
    _same_in_a_new_thread(lambda: moe.route_scored(z, 6))
    _same_in_a_new_thread(lambda: (moe.route_scored_backward(dg, z, idx),))


def test_combine_backward():
    dout, y, gate = _rand(1, 40, 256), _rand(2, 80, 256), _rand(3, 40, 2, dtype=F32)
    row_of = torch.randperm(80, device="cuda").to(torch.int32)
    _same_in_a_new_thread(lambda: moe.combine_backward(dout, y, row_of, gate))


def test_layer_and_its_steps():
    wl = synth.small("threads", 200, 256, 128, 4, 2)
    inp = synth.make_inputs(wl, "cuda")
    ws = moe.alloc_workspace(wl.T, wl.d, wl.f, wl.E, wl.k)
    w = inp["W1"], inp["W3"], inp["W2"]
    idx, gate = moe.route(inp["logits"], wl.k, ws)
    _, offsets, _, row_of, xp = moe.permute(inp["x"], idx, wl.E, ws)
    y = moe.grouped_ffn(xp, offsets, *w, wl.T, wl.k, ws)[1]
    _same_in_a_new_thread(lambda: moe.route(inp["logits"], wl.k, ws))
    _same_in_a_new_thread(lambda: moe.permute(inp["x"], idx, wl.E, ws))
    _same_in_a_new_thread(lambda: moe.grouped_ffn(xp, offsets, *w, wl.T, wl.k, ws))
    _same_in_a_new_thread(lambda: (moe.combine(y, row_of, gate),))
    _same_in_a_new_thread(lambda: (moe.layer_forward(inp["x"], inp["logits"], *w, wl.k, ws),))
    logits = inp["logits"]
    router = moe.Router(score=moe.SCORE_SIGMOID)
    _same_in_a_new_thread(lambda: (moe.layer_forward(inp["x"], logits, *w, wl.k, ws, router=router),))
