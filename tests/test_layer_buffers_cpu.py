"""Lifetime of the layers' workspaces, without a GPU: none is given back, or
taken from memory that was given back, while queued or captured work may use it."""

import weakref

import pytest
import torch

from host_double import package


@pytest.fixture
def quiet(monkeypatch):
    """The package, and a list that notes each wait for the device; capturing[0]: whether a graph is being captured."""
    P = package(monkeypatch)
    waits, capturing = [], [False]
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: waits.append(device))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    return P, waits, capturing


def users(P):
    """Calls that take a workspace for so many tokens (blocks), by name."""
    import orthogonal_reparameterized_poetx_amd.layer as layer
    lay = P.PoetxLayer(512, 512, 64, "bf16", "cpu")
    pool = {}
    shared = [P.PoetxLayer(512, 512, 64, "bf16", "cpu", ws_pool=pool) for _ in range(2)]

    def build(n):
        layer.build_layer_blocks([lay] * n, "forward")
        return [t for k, t in layer._build_ws.items() if k[0] == lay.device][0]

    def chain(n):
        layer.chain_rule_layers([lay] * n, [(lay.thR, lay.thP)] * n)
        return [t for k, t in layer._chain_ws.items() if k[0] == lay.device][0]
    return dict(layer=lambda n: lay.workspace(P.OP_FORWARD, 100 * n),
                pool=lambda n: shared[n % 2].workspace(P.OP_FORWARD, 100 * n), build=build, chain=chain)


@pytest.mark.parametrize("kind", ["layer", "pool", "build", "chain"])
def test_replaced_workspaces(monkeypatch, quiet, kind):
    P, waits, capturing = quiet
    import orthogonal_reparameterized_poetx_amd.layer as layer
    monkeypatch.setattr(layer, "_build_ws", {})
    monkeypatch.setattr(layer, "_chain_ws", {})
    monkeypatch.setattr(P._lib, "poetx_build_block_sets", lambda *a, **k: None)
    monkeypatch.setattr(P._lib, "poetx_chain_rule_sets", lambda *a, **k: None)
    monkeypatch.setattr(P._lib, "build_workspace_bytes", lambda n, b: 1000 * n)
    monkeypatch.setattr(P._lib, "chain_workspace_bytes", lambda n, b: 1000 * n)
    use = users(P)[kind]
    first = weakref.ref(use(1))
    assert len(waits) == 1                      # no other stream's work in the memory it comes from
    assert use(1) is first() and len(waits) == 1
    second = weakref.ref(use(2))
    assert len(waits) == 2 and first() is None  # done with by the time it is given back
    capturing[0] = True
    assert use(1) is second()
    capturing[0] = False
    third = weakref.ref(use(5))
    assert second() is not None                 # a graph holds it
    capturing[0] = True
    n = len(waits)
    fourth = weakref.ref(use(9))                # (a capture cannot wait: the smaller one stays)
    capturing[0] = False
    use(12)
    assert len(waits) == n + 1 and None not in (second(), third(), fourth())


def test_merge_takes_its_workspace_from_its_stream(monkeypatch, quiet):
    P, waits, _ = quiet
    made = []
    lay = P.PoetxLayer(512, 512, 64, "bf16", "cpu")
    monkeypatch.setattr(P._lib, "make_workspace", lambda *a: made.append(a))
    monkeypatch.setattr(P._lib, "poetx_merge_blocks_sets", lambda *a: None)
    P.merge_layers_sets([lay], stream="a stream")
    assert made[0][2] == "a stream"
