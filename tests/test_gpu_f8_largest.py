"""The largest magnitudes a cache in 8 bits can hold: blocks of 2^120, whose
codes from 256 on stand for 2^128 and more and are read as infinities, and the
blocks below. A value that a token does not see has no influence on it, however
large."""

from __future__ import annotations

import pytest
import torch

import f8_ref as F
import w4a4_linear_layers_amd as S
from test_gpu_f8_cache import DEV, INF, gen, ints, random_cache

pytestmark = pytest.mark.gpu
TYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


def attend(q, k, v, ks, vs, n, old=0):
    cache = S.KvCacheF8(*[c.to(DEV) for c in (k, v, ks, vs)])
    pages = torch.arange(k.shape[0], dtype=torch.int32, device=DEV)[None]
    return S.attn_prefill(q.to(DEV), ints([0, n]).to(DEV), cache, pages, ints([old + n]).to(DEV), max_len=old + n)


@TYPES
@pytest.mark.parametrize("D,Hq,Hkv,n,old,at", [(64, 2, 1, 40, 0, 37), (128, 8, 2, 90, 0, 70), (128, 4, 4, 20, 150, 165),
                                               (64, 4, 1, 300, 0, 64), (128, 1, 1, 17, 0, 16)])
@pytest.mark.parametrize("code", [0x77, 0x78, 0x7E, 0xF8, 0xFE])
def test_a_value_not_seen_however_large(dtype, D, Hq, Hkv, n, old, at, code):
    """Token `at` of a block of 2^120 has this code in keys and values: tokens before it come out bit for bit as
    with zeros there."""
    g = gen(n + code)
    pages = -(-(n + old) // 16)
    k, ks = random_cache(g, pages, Hkv, 16, D)
    v, vs = random_cache(g, pages, Hkv, 16, D)
    q = torch.randn(n, Hq, D, generator=g).to(dtype)
    p, t = at // 16, at % 16
    for c, s in ((k, ks), (v, vs)):
        s[p] = 247
        c.view(torch.uint8)[p] = 0
    clean = attend(q, k, v, ks, vs, n, old)
    for c in (k, v):
        c.view(torch.uint8)[p, :, t, ::3] = code
    got = attend(q, k, v, ks, vs, n, old)
    assert torch.isfinite(clean).all()
    assert torch.equal(got[:at - old], clean[:at - old])


@TYPES
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_number_stored_behind_the_mask(dtype, sign):
    """Stored by the append itself: tokens of earlier blocks come out as if it were small."""
    D, Hq, Hkv, n, at = 128, 4, 2, 60, 50
    g = gen(4)
    x = torch.randn(n, (Hq + 2 * Hkv) * D, generator=g).to(dtype)
    out = []
    for top in (1.0, sign * torch.finfo(dtype).max):
        x.view(n, -1, D)[at, Hq:, ::2] = top
        cache = S.KvCacheF8.empty(4, Hkv, 16, D)
        for c in (cache.k, cache.v, cache.k_scale, cache.v_scale):
            c.view(torch.uint8).fill_(0x30)
        slot = torch.arange(n, dtype=torch.int32, device=DEV)
        q = S.rope_append(x.to(DEV), Hq, cache, None, slot, None)
        pages = torch.arange(4, dtype=torch.int32, device=DEV)[None]
        out.append(S.attn_prefill(q, ints([0, n]).to(DEV), cache, pages, ints([n]).to(DEV), max_len=n))
    assert int(cache.v_scale[3, 0, 0]) == 247
    assert torch.isfinite(out[0]).all() and torch.equal(out[0][:48], out[1][:48])


@TYPES
def test_every_code_of_the_largest_scales(dtype):
    """One key: the output is the value itself, infinities from 2^128 on."""
    D, Hkv = 64, 4
    codes = torch.arange(256, dtype=torch.uint8).view(1, 4, 1, 64).repeat(1, 1, 16, 1)
    codes[codes == 127] = 0
    codes[codes == 255] = 0
    codes = codes.view(F.F8)
    zeros = torch.zeros(1, Hkv, 16, D, dtype=torch.uint8).view(F.F8)
    q = torch.zeros(1, Hkv, D, dtype=dtype, device=DEV)
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    for byte in range(240, 248):
        s = torch.full((1, Hkv, 1), byte, dtype=torch.uint8)
        cache = S.KvCacheF8(*[c.to(DEV) for c in (zeros, codes, s, s)])
        want = F.values(codes, s)[0, :, 0]
        want = torch.where(want.abs() >= 2.0 ** 128, want.sign() * INF, want)
        assert bool(torch.isinf(want).any()) == (byte == 247)
        for o in (S.attn_decode(q, cache, one[:, None] * 0, one, max_len=1),
                  S.attn_prefill(q, ints([0, 1]).to(DEV), cache, one[:, None] * 0, one, max_len=1)):
            got = o[0].double().cpu()
            assert torch.equal(got, want), (byte, got[got != want][:5], want[got != want][:5])
