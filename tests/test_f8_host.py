"""The cache in 8 bits without a GPU: refusals, which come before anything is
launched, workspace sizes, the binding's checks, and the tests' own plain forms."""

from __future__ import annotations

import ctypes
import math

import pytest
import torch

import f8_ref as F
import w4a4_linear_layers_amd as S
from w4a4_linear_layers_amd import _lib

A = 0x100000          # an aligned fake device address, never dereferenced
OK, EINVAL, EALIGN, EUNSUP = _lib.SERQ_OK, _lib.SERQ_EINVAL, _lib.SERQ_EALIGN, _lib.SERQ_EUNSUPPORTED
BF16, F32 = _lib.SERQ_BF16, _lib.SERQ_F32
AXES = bytes([0] * 16 + [1] * 24 + [2] * 24)


def append(f8, QKV=A, dt=BF16, ld=768, M=4, Hq=4, Hkv=1, D=128, qn=A, kn=A, eps=1e-5, table=A, rot=128, max_pos=10,
           layout=0, n_axes=3, axes=AXES, pos=A, slot=A, Q=A, ldq=512, Kc=A, Vc=A, ks=A, vs=A, n_pages=4, page=16):
    head = (QKV, dt, ld, M, Hq, Hkv, D, qn, kn, eps, table, rot, max_pos, layout, n_axes, axes, pos, slot, Q, ldq, Kc, Vc)
    if f8:
        return _lib.lib.serq_rope_append_f8(*head, ks, vs, n_pages, page, None)
    return _lib.lib.serq_rope_append_axes(*head, n_pages, page, None)


BOTH = [
    (dict(dt=2), EINVAL), (dict(layout=2), EINVAL), (dict(M=-1), EINVAL), (dict(Hkv=0), EINVAL), (dict(Hq=3, Hkv=2), EINVAL),
    (dict(D=96), EUNSUP), (dict(page=8), EUNSUP), (dict(page=24), EUNSUP), (dict(n_pages=0), EINVAL), (dict(n_pages=1 << 27), EINVAL),
    (dict(ld=767), EINVAL), (dict(ldq=511), EINVAL), (dict(rot=3), EINVAL), (dict(rot=130), EINVAL), (dict(table=None), EINVAL),
    (dict(eps=math.nan), EINVAL), (dict(Kc=None), EINVAL), (dict(Vc=None), EINVAL), (dict(QKV=None), EINVAL),
    (dict(slot=None), EINVAL), (dict(pos=None), EINVAL), (dict(Q=None), EINVAL), (dict(Kc=A + 8), EALIGN), (dict(Vc=A + 2), EALIGN),
    (dict(n_axes=0), EINVAL), (dict(n_axes=5), EINVAL), (dict(n_axes=2), EINVAL), (dict(axes=None), EINVAL),
    (dict(axes=bytes([3]) + AXES[1:]), EINVAL), (dict(axes=AXES[:-1] + bytes([255])), EINVAL),
    (dict(M=0), OK), (dict(M=0, QKV=None, slot=None, pos=None, Q=None), OK), (dict(M=0, n_axes=1, axes=None), OK),
    (dict(M=0, rot=0, table=None, max_pos=0, axes=None), OK), (dict(M=0, n_axes=4), OK),
]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("kw,code", BOTH)
def test_append_refusals(f8, kw, code):
    assert append(f8, **kw) == code


@pytest.mark.parametrize("kw,code", [(dict(ks=None), EINVAL), (dict(vs=None), EINVAL), (dict(ks=A + 2), EALIGN), (dict(vs=A + 1), EALIGN)])
def test_append_refuses_scales(kw, code):
    assert append(True, **kw) == code


def prefill(Q=A, dt=BF16, ldq=512, cu=A, B=2, T=9, Hq=4, Hkv=1, D=128, K=A, V=A, ks=A, vs=A, n_pages=4, page=16, table=A,
            max_pages=4, kv=A, max_len=64, scale=0.1, O=A, ldo=512, ws=None, size=0):
    return _lib.lib.serq_attn_prefill_f8(Q, dt, ldq, cu, B, T, Hq, Hkv, D, K, V, ks, vs, n_pages, page, table, max_pages, kv,
                                         max_len, scale, O, ldo, ws, size, None)


def decode(Q=A, dt=BF16, ldq=512, B=2, Hq=4, Hkv=1, D=128, K=A, V=A, ks=A, vs=A, n_pages=4, page=16, prefix=A, prefix_len=20,
           table=A, max_pages=4, kv=A, max_len=64, scale=0.1, O=A, ldo=512, ws=A, size=1 << 30):
    return _lib.lib.serq_attn_decode_f8(Q, dt, ldq, B, Hq, Hkv, D, K, V, ks, vs, n_pages, page, prefix, prefix_len, table,
                                        max_pages, kv, max_len, scale, O, ldo, ws, size, None)


@pytest.mark.parametrize("call", [prefill, decode])
@pytest.mark.parametrize("kw,code", [
    (dict(dt=7), EINVAL), (dict(B=-1), EINVAL), (dict(Hq=3, Hkv=2), EINVAL), (dict(D=80), EUNSUP), (dict(page=17), EUNSUP),
    (dict(max_len=(1 << 30) + 1), EINVAL), (dict(scale=math.inf), EINVAL), (dict(ldq=516), EALIGN), (dict(dt=F32, ldo=514), EALIGN),
    (dict(K=None), EINVAL), (dict(V=None), EINVAL), (dict(K=A + 8), EALIGN), (dict(ks=None), EINVAL), (dict(vs=None), EINVAL),
    (dict(ks=A + 1), EALIGN), (dict(vs=A + 2), EALIGN), (dict(Q=None), EINVAL), (dict(kv=None), EINVAL), (dict(table=None), EINVAL),
    (dict(B=0), OK), (dict(B=0, Q=None, O=None, kv=None, table=None), OK), (dict(B=0, ks=None), EINVAL)])
def test_attention_refusals(call, kw, code):
    assert call(**kw) == code


def test_workspaces_are_asked_for():
    assert prefill(max_len=100000, max_pages=1 << 20) == EINVAL and decode(ws=None) == EINVAL and decode(size=64) == EINVAL
    assert decode(ws=A + 4) == EALIGN
    p, d = _lib.lib.serq_attn_prefill_f8_workspace, _lib.lib.serq_attn_decode_f8_workspace
    assert p(BF16, 0, 0, 4, 1, 128, 100) == 0 and d(BF16, 0, 4, 1, 128, 0, 100) == 0
    assert p(BF16, 1, 4, 4, 3, 128, 100) == -1 and p(5, 1, 4, 4, 1, 128, 100) == -1 and p(BF16, 1, 4, 4, 1, 96, 1) == -1
    assert d(BF16, 1, 4, 1, 128, -1, 100) == -1 and d(BF16, -1, 4, 1, 128, 0, 100) == -1
    for dt in (BF16, F32):
        for b in (1, 3, 64, 500):
            for n in (0, 1, 127, 128, 129, 5000, 1 << 20, 1 << 30):
                assert 0 <= d(dt, b, 64, 8, 128, n, n) < 1 << 33


def cpu_cache(pages=2, Hkv=1, page=32, D=64):
    k = torch.zeros(pages, Hkv, page, D, dtype=F.F8)
    s = torch.zeros(pages, Hkv, page // 16, dtype=torch.uint8)
    return k, k.clone(), s, s.clone()


def test_binding_refuses_what_is_no_cache():
    k, v, ks, vs = cpu_cache()
    for bad in [(k, v, ks, vs),                                  # not on a device
                (k.float(), v, ks, vs), (k, v[:1], ks, vs), (k[0], v[0], ks, vs), (k, v, ks.int(), vs), (k, v, ks[..., :1], vs)]:
        with pytest.raises(ValueError):
            S.KvCacheF8(*bad)


# ------------------------------------------------------------------ the plain forms

def test_e4m3_is_torchs_rounding():
    g = torch.Generator()
    g.manual_seed(1)
    x = torch.cat([torch.randn(20000, generator=g) * 2.0 ** torch.randint(-14, 7, (20000,), generator=g),
                   torch.arange(256, dtype=torch.uint8).view(F.F8).float()[:127], torch.arange(0, 896) / 2.0 ** 13])
    x = torch.cat([x, (torch.arange(0, 3584) / 8.0).clamp(max=448)]).clamp(-448, 448)       # ties of every binade among them
    assert torch.equal(F.e4m3(x.double()), x.to(F.F8).double())


def test_exponent():
    for e in (-117, -100, -3, 0, 5, 120):
        top = 448.0 * 2.0 ** e
        assert F.exponent(top) == e and F.exponent(top * (1 + 2.0 ** -23)) == e + 1
        assert F.exponent(top / 2) == max(e - 1, -117) and F.exponent(top / 2 * (1 + 2.0 ** -23)) == e
    assert F.exponent(0.0) == -117 and F.exponent(1e-45) == -117


def test_addresses_reach_the_library_whole():
    assert ctypes.sizeof(ctypes.c_void_p) == 8 and len(_lib.lib.serq_rope_append_f8.argtypes) == 27
