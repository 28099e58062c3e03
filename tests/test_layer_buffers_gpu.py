"""A captured layer pass replays the same after larger eager calls have replaced its workspaces."""

import pytest

import workloads as WL
from gpu_util import make_layer, torch_mod

pytestmark = pytest.mark.gpu


def test_replay_after_a_larger_call():
    torch = torch_mod()
    inp = WL.small_case(91, 256, 512, 128, 40, dtype="bf16")
    lay, d = make_layer(inp)
    X = d["X"]
    dY = torch.randn(40, 256, device="cuda:0").to(torch.bfloat16)
    Y = lay.forward(X)
    dX, dR, dP = lay.backward(X, dY)
    want = [t.clone() for t in (Y, dX, dR, dP)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay.forward(X, Y)
        lay.backward(X, dY, dX=dX, dthR=dR, dthP=dP)
    big = torch.randn(5000, 512, device="cuda:0").to(torch.bfloat16)
    bigY = torch.randn(5000, 256, device="cuda:0").to(torch.bfloat16)
    for _ in range(3):
        lay.forward(big)
        lay.backward(big, bigY)
        held = [torch.full((1 << k,), float("nan"), device="cuda:0") for k in range(7, 22) for _ in range(6)]
        for t in (Y, dX, dR, dP):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (Y, dX, dR, dP)))
        assert all(bool(torch.isnan(t).all()) for t in held)
        del held
