"""The Python side of the linear in 8-bit integers on stand-in tensors (no GPU
needed): what it hands to the library, and what it refuses."""

from __future__ import annotations

import pytest
import torch

import w4a4_linear_layers_amd as S
from test_attention_binding import Fake, Recorder, floats


def codes(*shape):
    return Fake(*shape, dtype=torch.int8)


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(S, "lib", rec)
    monkeypatch.setattr(S, "_raw_stream", lambda device: 70 + device)
    monkeypatch.setattr(S, "_current_device", lambda: 0)
    return rec


def call(M=3, K=64, N=32, **kw):
    a = dict(xq=codes(M, K), sx=floats(M), Wq=codes(N, K), sw=floats(N), out=Fake(M, N))
    a.update(kw)
    layer = S.I8Layer(K=K, N=N, s_hat_inv=None, Wq=a.pop("Wq"), sw=a.pop("sw"))
    return S.linear_i8(a.pop("xq"), a.pop("sx"), layer, **a)


def test_what_is_handed_on(lib):
    call()
    assert lib.name == "serq_linear_i8" and lib.args[4:7] == (3, 64, 32) and lib.args[-1] == 70


@pytest.mark.parametrize("name,tensor", [("sx", lambda: floats(3)), ("sw", lambda: floats(32)), ("out", lambda: Fake(3, 32))])
def test_a_gradient_is_not_lost_silently(lib, name, tensor):
    t = tensor()
    t.requires_grad = True
    with pytest.raises(ValueError, match="gradient"):
        call(**{name: t})
    assert lib.name is None
    with torch.no_grad():
        call(**{name: t})
    assert t.address in lib.args
