"""Host checks of the optimizer entry points, and of the float64 reference's
8-bit format, without a GPU."""

import ctypes
import os

import numpy as np
import pytest

from oracle import operators as O


def _P():
    P = pytest.importorskip("orthogonal_reparameterized_poetx_amd")
    if not os.path.exists(P.LIB_PATH):
        pytest.skip("libpoetx.so not built")
    return P


def _param(P, **kw):
    d = dict(param=0x1000, grad=0x2000, copy_bf16=None, count=1000, lr_mul=1.0, weight_decay=0.0,
             param_dtype=P.POETX_F32, grad_dtype=P.POETX_F32)
    d.update(kw)
    return P.Param(*[d[k] for k, _ in P.Param._fields_])


def test_table_counts_and_layout():
    P = _P()
    host, s = P.param_table([_param(P, count=n) for n in (0, 1, 256, 257, 4096, 4097)])
    assert (s.blocks, s.values, s.count, s.norm_only) == (0 + 1 + 1 + 2 + 16 + 17, 8707, 6, 0)
    assert s.chunks >= 6 and not s.table and host.numel() >= 256 + 6 * 32
    assert not host[:256].any()         # the norm's arrival counter starts at zero
    _, s = P.param_table([_param(P, param=None)])
    assert s.norm_only == 1
    _, s = P.param_table([])
    assert s.blocks == s.chunks == 0


@pytest.mark.parametrize("kw,code", [(dict(count=-1), -2), (dict(count=(1 << 37) + 1), -2), (dict(param_dtype=5), -3),
                                     (dict(grad_dtype=-1), -3), (dict(grad=None), -1), (dict(grad=0x2002), -1),
                                     (dict(param=0x1001, param_dtype=1), -1), (dict(copy_bf16=0x3001), -1),
                                     (dict(copy_bf16=0x3000, param_dtype=1), -3)])
def test_table_refusals(kw, code):
    P = _P()
    arr = (P.Param * 2)(_param(P), _param(P, **kw))
    assert P.lib().poetx_param_table_bytes(arr, 2) == 0 and "tensor 1" in P.last_error() or "2^37" in P.last_error()
    buf, out = (ctypes.c_char * 4096)(), P.ParamSet()
    assert P.lib().poetx_param_table(arr, 2, ctypes.cast(buf, ctypes.c_void_p), 4096, ctypes.byref(out)) == code


def test_call_refusals():
    P = _P()
    L = P.lib()
    _, s = P.param_table([_param(P)])
    hp = P.AdamwHyper(1e-3, 0.9, 0.999, 1e-8)
    st = P.AdamwState(0x1000, 0x2000, 0x3000, 0x4000, P.POETX_STATE_8BIT, 0)
    r = ctypes.byref

    def step(pset=s, state=st, hyper=hp, n=1):
        return L.poetx_adamw_step(r(pset), r(state), r(hyper), n, None, None)
    assert step() == -1 and "table" in P.last_error()       # table not on the device
    s.table = 0x1010
    assert step() == -1                                     # not aligned
    s.table = 0x1000
    assert step(n=0) == -1
    for bad in (P.AdamwHyper(1e-3, 1.0, 0.999, 1e-8), P.AdamwHyper(1e-3, 0.9, -0.1, 1e-8),
                P.AdamwHyper(1e-3, 0.9, float("nan"), 1e-8), P.AdamwHyper(1e-3, 0.9, 0.999, -1.0)):
        assert step(hyper=bad) == -1
    for bad in (P.AdamwState(0x1000, 0x2000, None, 0x4000, 1, 0), P.AdamwState(None, 0x2000, None, None, 0, 0),
                P.AdamwState(0x1008, 0x2000, 0x3000, 0x4000, 1, 0), P.AdamwState(0x1000, 0x2000, 0, 0, 2, 0),
                P.AdamwState(0x1000, 0x2000, 0x3000, 0x4000, 1, 1)):
        assert step(state=bad) == -1
    assert L.poetx_adamw_step(None, r(st), r(hp), 1, None, None) == -1
    assert L.poetx_adamw_step(r(s), None, r(hp), 1, None, None) == -1
    assert L.poetx_adamw_step(r(s), r(st), None, 1, None, None) == -1
    only = P.ParamSet(0x1000, s.blocks, s.chunks, s.values, s.count, 1)
    assert step(pset=only) == -1 and "no param" in P.last_error()
    ws = P.grad_norm_workspace_bytes(s)
    fake = ctypes.c_void_p(0x1000)
    assert L.poetx_grad_norm(r(s), 0.0, fake, fake, ws, None) == -1
    assert L.poetx_grad_norm(r(s), float("nan"), fake, fake, ws, None) == -1
    assert L.poetx_grad_norm(r(s), 1.0, None, fake, ws, None) == -1
    assert L.poetx_grad_norm(r(s), 1.0, fake, fake, ws - 1, None) == -4
    assert L.poetx_grad_norm(r(s), 1.0, fake, None, ws, None) == -4
    assert L.poetx_adamw_moments(r(s), r(P.AdamwState(0x1000, 0x2000, None, None, 0, 0)), fake, fake, None) == -1
    assert L.poetx_adamw_moments(r(s), r(st), ctypes.c_void_p(0x1008), fake, None) == -1


def test_reference_rounding_of_8_bits_is_unbiased_and_invertible():
    rng = np.random.default_rng(2)
    x = rng.standard_normal(4 * O.BLOCK) * 10.0 ** rng.uniform(-3, 0, 4 * O.BLOCK)
    pos = np.arange(x.size)
    for signed, a in ((True, x), (False, x * x)):
        mean = np.zeros_like(a)
        for step in range(1, 513):
            r, unit = O.round8(a, pos, step, signed)
            assert np.all(np.abs(r - a) <= unit)
            mean += r / 512
        # a Weyl sequence of 512 terms misses a mean by O(log(512) / 512) of a step
        # (a second moment below the lowest step is kept at that step, not at zero)
        low = (a < unit) & (not signed)
        assert np.max((np.abs(mean - a) / unit)[~low]) <= 0.02
        assert np.allclose(mean[low], unit[low])
    # every code of a block decodes to a value that rounds to itself
    codes = np.arange(256)
    for signed in (True, False):
        val = O.decode8(codes, [130], signed)
        val = np.where(val == 0, 0.0, val)
        again, _ = O.round8(val, np.arange(256), 7, signed)
        assert np.array_equal(again, val)


def test_count_of_skipped_steps_is_checked():
    P = _P()
    _, s = P.param_table([_param(P)])
    s.table = 0x1000
    hp = P.AdamwHyper(1e-3, 0.9, 0.999, 1e-8)
    st = P.AdamwState(0x1000, 0x2000, 0x3000, 0x4000, P.POETX_STATE_8BIT, 0, 0x5002)
    r = ctypes.byref
    assert P.lib().poetx_adamw_step(r(s), r(st), r(hp), 1, None, None) == -1 and "skipped" in P.last_error()
    # the states of callers that do not know the field have none
    assert not P.AdamwState(0x1000, 0x2000, 0x3000, 0x4000, P.POETX_STATE_8BIT, 0).skipped
