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


@pytest.mark.parametrize("sizes", [dict(M=(1 << 32) + 5, K=1, N=1), dict(M=1 << 31, K=16, N=8), dict(K=(1 << 32) + 16, N=1), dict(N=(1 << 32) + 8, K=16)])
def test_sizes_that_no_int_holds_are_refused(lib, monkeypatch, sizes):
    """(ctypes would hand on their low 32 bits)"""
    with pytest.raises(ValueError):
        call(**sizes)
    assert lib.name is None
    monkeypatch.undo()
    M, K, N = ({**dict(M=3, K=64, N=32), **sizes}[k] for k in "MKN")
    assert S.linear_i8_workspace(M, K, N) == -1 and S.i8_kernel_name(M, K, N) is None


def test_sizes_are_told_from_those_of_other_bits():
    for sizes in ((-(1 << 32) + 3, 64, 32), (3, -(1 << 32) + 64, 32), (3, 64, -(1 << 32) + 32), (-1, 64, 32), (3, 0, 32), (3, 64, 0)):
        assert S.linear_i8_workspace(*sizes) == -1 and S.i8_kernel_name(*sizes) is None
    assert S.linear_i8_workspace(3, 64, 32) == 0 and S.i8_kernel_name(3, 64, 32) == "stream"
