"""A stand-in for device tensors, for tests of the classes' own bookkeeping
without a GPU (not collected by pytest): tensors in host memory that call
themselves device tensors, and a stream without work.  Nothing is launched; a
test replaces the library calls that would."""

import os

import pytest
import torch


class OnHost(torch.Tensor):
    is_cuda = property(lambda self: True)


def dev(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnHost)


class Stream:
    cuda_stream = 0

    def synchronize(self):
        pass


def package(monkeypatch):
    P = pytest.importorskip("orthogonal_reparameterized_poetx_amd")
    if not os.path.exists(P.LIB_PATH):
        pytest.skip("libpoetx.so not built")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    monkeypatch.setattr(P._lib, "stream_handle", lambda stream: 0)
    return P
