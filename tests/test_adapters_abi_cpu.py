"""Host checks of the adapter entry points without a GPU."""

import ctypes
import os

import pytest


def _P():
    P = pytest.importorskip("orthogonal_reparameterized_poetx_amd")
    if not os.path.exists(P.LIB_PATH):
        pytest.skip("libpoetx.so not built")
    return P


def _set(P, ranks=(16, 8), m=512, n=256, dtype=None, base=0x10000, **kw):
    rows = [P.Adapter(base, base, kw.get("dA"), kw.get("dB"), r, 1.0) for r in ranks]
    _, s = P.adapter_table(rows, m, n, P.POETX_BF16 if dtype is None else dtype)
    s.table = 0x1000
    return s


def test_table():
    P = _P()
    s = _set(P)
    assert (s.m, s.n, s.count, s.max_rank, s.rows, s.layout, s.flags) == (512, 256, 2, 16, 32, 3, 0)
    assert _set(P, (16, 40, 3)).rows == 32 + 64 + 32           # whole matrix steps of 32 once a rank exceeds 16
    assert _set(P, (16, 5)).layout == 1 and _set(P, n=260).layout == 2 and _set(P, base=0x10002).layout == 0
    assert _set(P, (4,), n=260, dtype=P.POETX_F32).layout == 3
    assert _set(P, ()).count == 0


@pytest.mark.parametrize("kw,code", [(dict(ranks=(0,)), -2), (dict(ranks=(257,)), -2), (dict(m=0), -2),
                                     (dict(n=32769), -2), (dict(dtype=3), -3), (dict(base=None), -1),
                                     (dict(base=0x10001), -1), (dict(base=0x10002, dtype=0), -1),
                                     (dict(dA=0x10002), -1), (dict(dB=0x10001), -1)])
def test_table_refusals(kw, code):
    P = _P()
    with pytest.raises(P.PoetxError) as e:
        _set(P, **kw)
    assert e.value.code == code


def test_call_refusals():
    P = _P()
    L = P.lib()
    s = _set(P)
    f = ctypes.c_void_p(0x10000)
    r = ctypes.byref
    need = P.adapters_workspace_bytes(s, 100, 3, P.OP_FORWARD)
    bneed = P.adapters_workspace_bytes(s, 100, 3, P.OP_BACKWARD)
    assert 0 < need < bneed
    assert L.poetx_adapters_workspace_bytes(r(s), 100, 3, P.OP_MERGE) == 0
    assert L.poetx_adapters_workspace_bytes(r(s), -1, 3, 0) == 0

    def fwd(aset=s, start=f, which=f, nseg=3, X=f, ldx=256, N=100, Y=f, ldy=512, ws=f, nbytes=need):
        return L.poetx_adapters_forward(r(aset), start, which, nseg, X, ldx, N, Y, ldy, ws, nbytes, None)

    def bwd(aset=s, start=f, which=f, nseg=3, X=f, ldx=256, dY=f, lddy=512, N=100, dX=f, lddx=256, ws=f,
            nbytes=bneed):
        return L.poetx_adapters_backward(r(aset), start, which, nseg, X, ldx, dY, lddy, N, dX, lddx, ws, nbytes, None)
    odd = ctypes.c_void_p(0x10001)
    for call in (fwd, bwd):
        for kw, code in [(dict(start=None), -1), (dict(which=None), -1), (dict(nseg=-1), -2),
                         (dict(nseg=(1 << 20) + 1), -2), (dict(N=-1), -2), (dict(N=1 << 31), -2), (dict(X=None), -1),
                         (dict(X=odd), -1), (dict(ldx=255), -2), (dict(ws=None), -4),
                         (dict(ws=ctypes.c_void_p(0x10010)), -4), (dict(nbytes=16), -4)]:
            assert call(**kw) == code, (call, kw, P.last_error())
            assert P.last_error()
    assert fwd(Y=None) == -1 and fwd(ldy=511) == -2 and bwd(dY=None) == -1 and bwd(lddx=1) == -2
    for field, value in [("reserved", 1), ("max_rank", 0), ("max_rank", 300), ("count", -1), ("flags", 2),
                         ("layout", 8), ("table", None), ("table", 0x1010), ("rows", -1)]:
        t = _set(P)
        setattr(t, field, value)
        assert fwd(aset=t) == -1 and bwd(aset=t) == -1, field
    # empty calls enqueue nothing
    assert fwd(N=0) == 0 and fwd(nseg=0) == 0
    none = _set(P, ())
    assert fwd(aset=none) == 0 and bwd(aset=none) == 0


def test_workspace_goes_by_the_batch_not_by_the_set():
    """Partial sums of the gradients (rank x (m + n) fp32 each) are for the adapters that have tokens: a large set
    adds its transposed A (2 bytes, ranks padded to 16) and a few words an adapter."""
    P = _P()
    few, many = _set(P, (16,) * 4, m=1024, n=512), _set(P, (16,) * 4000, m=1024, n=512)
    for N, nseg in ((64, 4), (5000, 4), (64, 64)):
        extra = P.adapters_workspace_bytes(many, N, nseg, P.OP_BACKWARD) - \
            P.adapters_workspace_bytes(few, N, nseg, P.OP_BACKWARD)
        assert extra <= 4000 * (16 * 512 * 2 + 16) + nseg * 16 * (1024 + 512) * 4 + 4096, (N, nseg, extra)
