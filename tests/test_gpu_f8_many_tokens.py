"""Prompts of many tokens or heads onto a cache in 8 bits (from 2^16 tokens times
heads on keys and values take a launch of their own), in every form of the
rotation: both layouts, several axes, part of the head, rows that suit no vector
loads. Codes and scales bit for bit, queries those of a cache of the model's type."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import f8_ref as F
import w4a4_linear_layers_amd as S
from test_gpu_f8_cache import DEV, axes_of, gen, ints, random_cache

pytestmark = pytest.mark.gpu


def turned(x, w, eps, table, pos, listed, layout):
    """f8_ref.rotate, all rows at once. x: M x heads x D, pos: axes x M."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    if table is None:
        return x
    half = table.shape[1] // 2
    at = pos.long()[torch.tensor(listed)].t()                  # M x pairs: each pair's position
    i = torch.arange(half)
    c, s = (table.double()[at, i + o][:, None] for o in (0, half))
    y = x.clone()
    a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def test_the_plain_form_is_the_tests_other_one():
    g = gen(1)
    for layout, n, rot in (("half", 3, 22), ("interleaved", 2, 64), ("interleaved", 1, 6)):
        x, w = torch.randn(9, 2, 64, generator=g), torch.randn(64, generator=g)
        table = torch.randn(17, rot, generator=g)
        pos = torch.randint(0, 17, (n, 9), generator=g)
        listed = axes_of(rot, n, "turns")[1]
        a, b = turned(x, w, 1e-5, table, pos, listed, layout), F.rotate(x, w, 1e-5, table, pos, listed, layout)
        assert (a - b).abs().max() <= 1e-14 * b.abs().max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,Hkv,D,rot,norm,layout,axes,kind,pad,shift", [
    (2048, 8, 128, 128, True, "interleaved", 1, "blocks", 0, 0),
    (2051, 8, 64, 64, False, "interleaved", 1, "blocks", 0, 0),
    (2300, 8, 128, 64, True, "interleaved", 3, "turns", 0, 0),
    (2200, 8, 128, 128, True, "half", 3, "blocks", 0, 0),
    (2047, 8, 128, 128, True, "half", 3, "turns", 0, 0),       # (one launch)
    (4100, 9, 128, 128, True, "half", 3, "turns", 0, 0),       # (queries of three heads a lane)
    (4099, 5, 64, 64, True, "interleaved", 4, "blocks", 0, 0),
    (16500, 1, 64, 32, False, "half", 2, "turns", 0, 0),
    (2100, 1, 64, 32, False, "half", 2, "turns", 0, 0),        # (one launch)
    (120, 137, 128, 128, True, "half", 1, "blocks", 0, 0),     # few tokens of many heads
    (2600, 9, 128, 128, True, "half", 1, "blocks", 0, 0),
    (2050, 8, 64, 64, True, "half", 1, "blocks", 0, 0),
    (2070, 8, 64, 0, True, "half", 1, "blocks", 0, 0),
    (2071, 8, 128, 0, False, "half", 1, "blocks", 0, 0),
    (2049, 8, 128, 128, True, "half", 3, "turns", 1, 0),       # rows that lie unaligned
    (2500, 7, 64, 64, False, "interleaved", 2, "blocks", 0, 1),
    (2064, 8, 64, 20, True, "half", 3, "blocks", 0, 0),        # a part that no whole 16 bytes hold
    (2065, 8, 128, 6, True, "interleaved", 3, "turns", 8, 8),
])
def test_append(dtype, M, Hkv, D, rot, norm, layout, axes, kind, pad, shift):
    g = gen(M + rot)
    Hq, page = 2 * Hkv, 32
    slot, at, left = [], 0, M
    while left:                                                # prompts that begin and end inside blocks
        n = min(left, int(torch.randint(1, 500, (1,), generator=g)))
        lead = int(torch.randint(0, 16, (1,), generator=g))
        slot += range(at + lead, at + lead + n)
        at += -(-(n + lead) // page) * page
        left -= n
    pages = at // page
    width = (Hq + 2 * Hkv) * D
    flat = torch.randn(M * (width + pad) + shift, generator=g).to(dtype)
    qkv = torch.as_strided(flat, (M, width), (width + pad, 1), shift)
    dq = torch.as_strided(flat.to(DEV), (M, width), (width + pad, 1), shift)
    table = torch.from_numpy(S.rope_table(rot, 300, theta=900.0)) if rot else None
    pos = torch.randint(0, 300, (axes, M), generator=g).to(torch.int32)
    pair_axis, listed = axes_of(rot, axes, kind)
    w = 1 + 0.3 * torch.randn(D, generator=g) if norm else None
    k, s = random_cache(g, pages, Hkv, page, D)
    eps = float(np.float32(1e-6))
    kw = dict(layout=layout, eps=eps, q_norm=w.to(DEV) if norm else None, k_norm=w.to(DEV) if norm else None)
    if axes > 1:
        kw["pair_axis"] = pair_axis
    args = (pos if axes > 1 else pos[0]).to(DEV), ints(slot).to(DEV), table.to(DEV) if rot else None
    cache = S.KvCacheF8(*[c.to(DEV) for c in (k, k, s, s.clone())])
    q = S.rope_append(dq, Hq, cache, *args, **kw)
    x = qkv.reshape(M, -1, D)
    y = turned(x[:, Hq:Hq + Hkv], w, eps, table, pos, listed, layout).float().double()
    for name, want, c, cs in (("keys", y, cache.k, cache.k_scale), ("values", x[:, Hq + Hkv:].double(), cache.v, cache.v_scale)):
        codes, scale = F.store(k.double(), s, want, slot)
        assert torch.equal(cs.cpu(), scale), name
        F.same(c, codes, name)
    plain = S.KvCache(*[torch.zeros(pages, Hkv, page, D, dtype=dtype, device=DEV) for _ in range(2)])
    assert torch.equal(q, S.rope_append(dq, Hq, plain, *args, **kw))
