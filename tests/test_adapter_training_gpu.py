"""The operators together, as examples/train_adapters.py uses them: generators
and adapters trained by one clipped AdamW, 8-bit moments beside 32-bit ones, then
single tokens served."""

import importlib.util
import os

import numpy as np
import pytest

from gpu_util import torch_mod

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_adapters.py")


def example():
    spec = importlib.util.spec_from_file_location("train_adapters", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_training_and_serving():
    """The rank-16 adapters can express the rank-4 teachers: the loss falls to a tenth within 150 steps, with 8-bit
    moments as with 32-bit ones (twice the final loss is allowed), and tokens served alone equal those of whole
    segments to the rounding of bf16 outputs (2^-7 of the value, plus that of T's order of summation, 1e-3)."""
    torch = torch_mod()
    ex = example()
    final = {}
    for bits in (32, 8):
        model, losses = ex.train(steps=150, width=256, tasks=3, rank=16, state_bits=bits)
        assert np.all(np.isfinite(losses))
        final[bits] = np.mean(losses[-10:])
        assert final[bits] < 0.1 * losses[0], losses[::15]
        for half, whole in zip(model.adapters.A + model.adapters.B, model.opt.params[2:]):
            assert torch.equal(half, whole.to(torch.bfloat16))      # the copies follow the master values
        assert bool(model.layer.thR.any())
        one, whole = ex.serve(model)
        d = (one.float() - whole.float()).abs()
        assert bool((d <= 2.0 ** -7 * whole.float().abs() + 1e-3).all())
    assert final[8] < 2 * final[32]


def test_the_layers_results_do_not_change():
    """A layer without adapters, and one whose segments have none, give the same bits."""
    torch = torch_mod()
    ex = example()
    model = ex.Model(256, 2, 8, 8)
    X = torch.randn(100, 256, device="cuda:0").to(torch.bfloat16)
    plain = model.layer.forward(X)
    seg = ex.segments([40, 60], [-1, -1], "cuda:0")
    assert torch.equal(model.adapters.forward(X, model.layer.forward(X), *seg), plain)
