"""What AdapterSet and AdamW hand to the library: checks of the caller's buffers
and lifetime of their own, without a GPU."""

import contextlib
import weakref

import pytest
import torch

from host_double import OnHost, dev, package


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


class Side:
    def __init__(self, handle):
        self.cuda_stream, self.waits = handle, []

    def synchronize(self):
        pass

    def wait_stream(self, other):
        self.waits.append(other)


class External(Side):
    pass


def streams(monkeypatch):
    """The package, the streams that each buffer is recorded on, and the stream that each workspace is made on."""
    P = package(monkeypatch)
    current, recorded, made, context = Side(0), [], {}, [None]
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(P._lib, "stream_handle",
                        lambda s: 0 if s is None else s if isinstance(s, int) else s.cuda_stream)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s.cuda_stream)))
    monkeypatch.setattr(P._lib, "poetx_adapters_forward", lambda *a: None)
    monkeypatch.setattr(P._lib, "poetx_adapters_backward", lambda *a: None)
    monkeypatch.setattr(P._lib, "poetx_adamw_step", lambda *a: None)
    monkeypatch.setattr(P._lib, "poetx_grad_norm", lambda *a: None)
    monkeypatch.setattr(P._lib, "poetx_adamw_moments", lambda *a: None)

    @contextlib.contextmanager
    def on(s):
        context.append(s)
        yield
        context.pop()
    monkeypatch.setattr(torch.cuda, "stream", on)
    real = torch.empty

    def note(*a, **kw):
        t = real(*a, **kw).as_subclass(OnHost)
        made[t.data_ptr()] = context[-1] and context[-1].cuda_stream
        return t
    monkeypatch.setattr(torch, "empty", note)
    return P, current, recorded, made


def test_buffers_of_an_adapter_set_know_their_streams(monkeypatch):
    P, current, recorded, made = streams(monkeypatch)
    s = adapters(P)
    X, Y = dev(40, 256, dtype=torch.bfloat16), dev(40, 512, dtype=torch.bfloat16)
    seg = dev(2, dtype=torch.int32), dev(1, dtype=torch.int32)
    a = Side(7)
    s.forward(X, Y, *seg, stream=a)
    ws = s.workspace(P.OP_FORWARD, 40, 1)
    # made where it is first used: the current stream's queued work may still hold what it gave back
    assert made[ws.data_ptr()] == 7
    assert (s.table.data_ptr(), 7) in recorded
    # used on a second stream
    s.forward(X, Y, *seg)
    assert (ws.data_ptr(), 0) in recorded
    n = len(recorded)
    for _ in range(3):
        s.forward(X, Y, *seg)
        s.forward(X, Y, *seg, stream=a)
    assert len(recorded) == n            # known: nothing more to do
    # a workspace that is made later knows both
    s.backward(X, Y, *seg, stream=a)
    wb = s.workspace(P.OP_BACKWARD, 40, 1)
    assert made[wb.data_ptr()] == 7 and (wb.data_ptr(), 0) in recorded
    # a raw handle may be gone when the buffers are given back: made there, not recorded
    s.forward(dev(4000, 256, dtype=torch.bfloat16), dev(4000, 512, dtype=torch.bfloat16), *seg, stream=9)
    ws = s.workspace(P.OP_FORWARD, 4000, 1)
    assert made[ws.data_ptr()] == 9 and not [r for r in recorded if r[1] == 9]
    s.forward(X, Y, *seg, stream=External(9))
    assert not [r for r in recorded if r[1] == 9]
    # the same stream, now as one of torch's own: known from here on
    s.forward(X, Y, *seg, stream=Side(9))
    assert {(t.data_ptr(), 9) for t in (s.table, ws, wb)} <= set(recorded)


def test_buffers_of_the_optimizer_know_their_streams(monkeypatch):
    P, current, recorded, made = streams(monkeypatch)
    a = Side(7)
    opt = adamw(P, 300, 8)
    opt.step(stream=a)
    assert {(t.data_ptr(), 7) for t in [opt.table, *opt.state().values()]} <= set(recorded)
    norm = P.GradNorm([dev(300)])
    norm(1.0, stream=a)
    assert {(t.data_ptr(), 7) for t in (norm.table, norm.ws, norm.out)} <= set(recorded)
    # outputs made for another stream's call: it waits for the work of the stream they come from
    m, v = opt.moments(stream=a)
    assert a.waits == [current] and {(m.data_ptr(), 7), (v.data_ptr(), 7)} <= set(recorded)
    opt.moments()
    assert a.waits == [current]
    e = External(9)
    opt.moments(stream=e)
    assert e.waits == [current] and not [r for r in recorded if r[1] == 9]


def test_tensors_of_the_table_live_as_long_as_the_object(monkeypatch):
    """The table holds their addresses, whatever becomes of the caller's lists."""
    P = package(monkeypatch)
    state = dict(m=dev(256), v=dev(256))
    p, g, c = [dev(200)], [dev(200)], [dev(200, dtype=torch.bfloat16)]
    refs = [weakref.ref(t) for t in (p[0], g[0], c[0])]
    opt = P.AdamW(p, g, copies=c, state=state)
    norm = P.GradNorm(g)
    for ts in (p, g, c, opt.params, opt.grads, norm.grads):
        ts.clear()
    assert all(r() is not None for r in refs)
    A, B, dA, dB = [dev(4, 64)], [dev(32, 4)], [dev(4, 64)], [dev(32, 4)]
    refs = [weakref.ref(t[0]) for t in (A, B, dA, dB)]
    s = P.AdapterSet(32, 64, A, B, [1.0], dA=dA, dB=dB)
    for ts in (A, B, dA, dB, s.A, s.B, s.dA, s.dB):
        ts.clear()
    assert all(r() is not None for r in refs)
    del opt, norm, s


def test_first_gradient_norm_makes_nothing(monkeypatch):
    """It may be inside a graph capture, which cannot wait for a stream."""
    P = package(monkeypatch)
    calls = []
    monkeypatch.setattr(P._lib, "poetx_grad_norm", lambda *a: calls.append(a))
    opt = adamw(P, 300, 8)
    for name in ("zeros", "empty"):
        monkeypatch.setattr(torch, name, lambda *a, **k: pytest.fail("a buffer is made"))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: pytest.fail("a stream is waited for"))
    monkeypatch.setattr(P._lib.Owned, "handle", lambda self, stream: 0)
    norm, coef = opt.grad_norm(1.0)
    assert len(calls) == 1 and norm.numel() == coef.numel() == 1
