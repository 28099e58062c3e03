"""What AdapterSet and AdamW hand to the library: checks of the caller's buffers
and lifetime of their own, without a GPU."""

import weakref

import pytest
import torch

from host_double import dev, package


def adamw(P, n, bits):
    """AdamW of one tensor, its moments in host memory too."""
    blocks = -(-n // 256)
    dt = torch.uint8 if bits == 8 else torch.float32
    state = dict(m=dev(blocks * 256, dtype=dt), v=dev(blocks * 256, dtype=dt))
    if bits == 8:
        state.update(m_exp=dev(blocks, dtype=dt), v_exp=dev(blocks, dtype=dt))
    return P.AdamW([dev(n)], [dev(n)], state_bits=bits, state=state)


@pytest.mark.parametrize("bad", [dict(n=255), dict(n=511), dict(dtype=torch.float32), dict(stride=2), dict(host=True)])
@pytest.mark.parametrize("which", [0, 1])
def test_moments_refuse_other_outputs(monkeypatch, bad, which):
    """A smaller or wider tensor would be written past its end, one of another type filled with foreign bits."""
    P = package(monkeypatch)
    calls = []
    monkeypatch.setattr(P._lib, "poetx_adamw_moments", lambda *a: calls.append(a))
    opt = adamw(P, 300, 8)          # two blocks of 256
    stride = bad.get("stride", 1)
    t = dev(bad.get("n", 512) * stride, dtype=bad.get("dtype", torch.bfloat16))[::stride]
    if "host" in bad:
        t = t.as_subclass(torch.Tensor)
    out = [dev(512, dtype=torch.bfloat16), t]
    with pytest.raises(ValueError):
        opt.moments(out=out[::-1] if which == 0 else out)
    with pytest.raises(ValueError):
        opt.moments(out=[dev(512, dtype=torch.bfloat16)])
    assert not calls
    good = [dev(2, 256, dtype=torch.bfloat16), None]
    assert opt.moments(out=good)[0] is good[0] and len(calls) == 1 and calls[0][2] is good[0]


def test_moments_of_32_bits_take_no_output(monkeypatch):
    P = package(monkeypatch)
    opt = adamw(P, 300, 32)
    assert opt.moments()[0].dtype == torch.float32
    with pytest.raises(ValueError):
        opt.moments(out=[dev(512), dev(512)])


def adapters(P, m=512, n=256, ranks=(16, 8), **kw):
    return P.AdapterSet(m, n, [dev(r, n, dtype=torch.bfloat16) for r in ranks],
                        [dev(m, r, dtype=torch.bfloat16) for r in ranks], [1.0] * len(ranks), **kw)


@pytest.mark.parametrize("op", ["OP_FORWARD", "OP_BACKWARD"])
def test_a_replaced_workspace_stays(monkeypatch, op):
    """A captured graph, or work queued on some stream, may still use the smaller one."""
    P = package(monkeypatch)
    s = adapters(P)
    op = getattr(P, op)
    live = []
    for N in (64, 65, 70, 100, 8192, 3000, 9000, 20000):
        ws = s.workspace(op, N, 3)
        assert ws.numel() >= P.adapters_workspace_bytes(s.aset, N, 3, op)
        live.append((weakref.ref(ws), ws.data_ptr()))
        assert s.workspace(op, 64, 3) is ws         # smaller calls take the one there is
        del ws
    assert all(r() is not None for r, _ in live)
    # what is kept is less than what is in use
    kept = {p: r().numel() for r, p in live}
    assert sum(kept.values()) < 2 * max(kept.values())
