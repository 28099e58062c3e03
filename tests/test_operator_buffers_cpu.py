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


def test_first_backward_leaves_the_table_where_it_is(monkeypatch):
    """A forward captured before it reads A and B through that table."""
    P = package(monkeypatch)
    seen = []
    monkeypatch.setattr(P._lib, "poetx_adapters_backward", lambda aset, *a: seen.append((aset.table, aset.flags)))
    s = adapters(P)
    where, before = s.aset.table, s.table.clone()
    assert where == s.table.data_ptr()
    X, dY = dev(40, 256, dtype=torch.bfloat16), dev(40, 512, dtype=torch.bfloat16)
    seg = dev(2, dtype=torch.int32), dev(1, dtype=torch.int32)
    dA, dB = s.backward(X, dY, *seg)
    assert s.table.data_ptr() == where and seen == [(where, 0)]
    # the same pointers of A and B, now with gradients
    rows = [t.view(torch.int64).view(len(dA), -1) for t in (before, s.table)]
    assert torch.equal(rows[0][:, :2], rows[1][:, :2]) and not rows[0][:, 2:4].any()
    assert rows[1][:, 2].tolist() == [t.data_ptr() for t in dA] and rows[1][:, 3].tolist() == [t.data_ptr() for t in dB]
    s.backward(X, dY, *seg, accumulate=True)
    assert seen[1:] == [(where, P.POETX_ACCUMULATE_GRAD)]


def test_first_backward_inside_a_capture_is_refused(monkeypatch):
    """It makes the gradients and copies the table from the host, which a capture cannot hold."""
    P = package(monkeypatch)
    seen = []
    monkeypatch.setattr(P._lib, "poetx_adapters_backward", lambda *a: seen.append(a))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    X, dY = dev(40, 256, dtype=torch.bfloat16), dev(40, 512, dtype=torch.bfloat16)
    seg = dev(2, dtype=torch.int32), dev(1, dtype=torch.int32)
    s = adapters(P)
    with pytest.raises(RuntimeError):
        s.backward(X, dY, *seg)
    assert s.dA is None and s.dB is None and not seen
    adapters(P, dA=[dev(16, 256), dev(8, 256)], dB=[dev(512, 16), dev(512, 8)]).backward(X, dY, *seg)
    assert len(seen) == 1
