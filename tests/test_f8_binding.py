"""The Python side of the calls on a cache in 8 bits, of positions on several
axes and of the linear in 8-bit integers, on stand-in tensors (no GPU needed):
what it hands to the library, and what it refuses."""

from __future__ import annotations

import pytest
import torch

import w4a4_linear_layers_amd as S
from test_attention_binding import CALLS, Fake, call_append, cache, floats, ints, lib  # noqa: F401

F8 = torch.float8_e4m3fn


def bytes_(*shape, device=0):
    return Fake(*shape, dtype=torch.uint8, device=device)


def cache8(device=0, pages=4):
    k, v = (Fake(pages, 2, 16, 64, dtype=F8, device=device) for _ in range(2))
    return S.KvCacheF8(k, v, bytes_(pages, 2, 1, device=device), bytes_(pages, 2, 1, device=device))


def handed(lib):
    """(k, v, k scale, v scale, pages, page size) of the last call."""
    a = lib.args
    return {"serq_rope_append_f8": a[20:26], "serq_attn_prefill_f8": a[9:15], "serq_attn_decode_f8": a[7:13]}[lib.name]


@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, 1), (torch.float32, 0)])
@pytest.mark.parametrize("call", CALLS)
def test_what_is_handed_on(lib, call, dtype, code):
    c = cache8()
    call(c, dtype=dtype)
    assert handed(lib) == (c.k.address, c.v.address, c.k_scale.address, c.v_scale.address, 4, 16) and lib.args[1] == code
    assert lib.args[-1] == 70
    c.k, c.k_scale, c.v, c.v_scale = (Fake(9, 2, 16, 64, dtype=F8), bytes_(9, 2, 1), Fake(9, 2, 16, 64, dtype=F8), bytes_(9, 2, 1))
    call(c, dtype=dtype)
    assert handed(lib) == (c.k.address, c.v.address, c.k_scale.address, c.v_scale.address, 9, 16)


@pytest.mark.parametrize("call", CALLS)
def test_kernels_are_launched_on_the_cache_s_device(lib, call):
    call(cache8(1), d=1)
    assert lib.on == 1 and lib.args[-1] == 71 and lib.current == 0


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("field,value", [
    ("k_scale", bytes_(4, 2, 2)), ("v_scale", ints(4, 2, 1)), ("k_scale", bytes_(4, 2, 1, device=1)),
    ("v", Fake(4, 2, 16, 64)), ("k", Fake(5, 2, 16, 64, dtype=F8)), ("v", Fake(4, 2, 16, 64, dtype=F8, device=1))])
def test_a_cache_replaced_in_part_is_refused(lib, call, field, value):
    c = cache8()
    setattr(c, field, value)
    with pytest.raises(ValueError):
        call(c)


@pytest.mark.parametrize("call", CALLS)
def test_a_gradient_is_not_lost_silently(lib, call):
    c = cache8()
    q = Fake(*((3, 8 * 64) if call is call_append else (2, 4, 64)))
    q.requires_grad = True
    with pytest.raises(ValueError):
        call(c, **({"qkv": q} if call is call_append else {"q": q}))


def test_queries_of_other_types_are_refused(lib):
    for call in CALLS:
        with pytest.raises(ValueError):
            call(cache8(), dtype=torch.float16)


@pytest.mark.parametrize("c", [cache, cache8])
def test_axes(lib, c):
    axes = [0] * 8 + [1] * 12 + [2] * 12
    for given in (axes, tuple(axes), bytes(axes), torch.tensor(axes)):
        call_append(c(), pair_axis=given, pos=ints(3, 3))
        assert lib.name == ("serq_rope_append_axes" if c is cache else "serq_rope_append_f8")
        assert lib.args[14] == 3 and bytes(lib.args[15]) == bytes(axes)
    call_append(c(), pair_axis=bytes(32), pos=ints(1, 3))
    assert lib.args[14] == 1
    for bad in (dict(pair_axis=axes, pos=ints(2, 3)), dict(pair_axis=axes[:-1], pos=ints(3, 3)), dict(pair_axis=axes, pos=ints(3)),
                dict(pair_axis=axes, pos=ints(3, 4)), dict(pair_axis=axes, pos=ints(5, 3)), dict(pair_axis=[300] * 32, pos=ints(3, 3)),
                dict(pair_axis=axes, pos=ints(3, 3, device=1))):
        with pytest.raises(ValueError):
            call_append(c(), **bad)


def test_axes_without_a_table_are_not_looked_at(lib):
    call_append(cache8(), table=None, pair_axis=[7], pos=None)
    assert lib.args[14] == 1 and lib.args[15] is None


def test_linear_refusals_name_no_device():
    """(host tensors, as far as the checks go without a GPU)"""
    layer = S.I8Layer(K=64, N=32, s_hat_inv=None, Wq=torch.zeros(32, 64, dtype=torch.int8), sw=torch.ones(32))
    x, sx = torch.zeros(3, 64, dtype=torch.int8), torch.ones(3)
    for args in ((x, sx, layer), (x.int(), sx, layer), (x[:, 1:], sx, layer),
                 (x, sx, S.I8Layer(K=32, N=32, s_hat_inv=None, Wq=layer.Wq, sw=layer.sw))):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            S.linear_i8(*args)
