"""What AdapterSet and AdamW hand to the library: checks of the caller's buffers
and lifetime of their own, without a GPU."""

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
