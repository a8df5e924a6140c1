"""The cache in 8 bits: serq_rope_append_f8, serq_attn_prefill_f8 and
serq_attn_decode_f8 against plain 64-bit forms (f8_ref.py, attention_ref.py),
and serq_rope_append_axes. Unused cache slots hold the code NaN, and unused
blocks a scale that is no number."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as R
import f8_ref as F
import w4a4_linear_layers_amd as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


def axes_of(rot, n, kind):
    """(pair_axis, its list): blocks of pairs, or axes taking turns."""
    half = rot // 2
    a = [i * n // half if kind == "blocks" else i % n for i in range(half)]
    return bytes(a), a


def random_cache(g, pages, Hkv, page, D):
    codes = (torch.randn(pages, Hkv, page, D, generator=g) * 60).clamp(-448, 448).to(F.F8)
    scale = torch.randint(115, 124, (pages, Hkv, page // 16), generator=g).to(torch.uint8)
    return codes, scale


# ------------------------------------------------------------------ append

def run_append(g, slots, Hq, Hkv, D, page, dtype, layout, rot, qn, kn, *, pages=None, axes=1, kind="blocks", pad=0, shift=0,
               gain=1.0):
    M = len(slots)
    width = (Hq + 2 * Hkv) * D
    flat = (torch.randn(M * (width + pad) + shift, generator=g) * gain).to(dtype)
    qkv = torch.as_strided(flat, (M, width), (width + pad, 1), shift)
    dq = torch.as_strided(flat.to(DEV), (M, width), (width + pad, 1), shift)
    max_pos = 97
    table = torch.from_numpy(S.rope_table(rot, max_pos, theta=1000.0)) if rot else None
    pos = torch.randint(0, max_pos, (axes, M), generator=g).to(torch.int32)
    pair_axis, listed = axes_of(rot, axes, kind)
    slot = ints(slots)
    pages = pages or max(slots + [0]) // page + 2
    w = [1 + 0.3 * torch.randn(D, generator=g) if f else None for f in (qn, kn)]
    start = [random_cache(g, pages, Hkv, page, D) for _ in range(2)]
    cache = S.KvCacheF8(*[c.to(DEV) for c in (start[0][0], start[1][0], start[0][1], start[1][1])])
    eps = float(np.float32(1e-5))
    q = S.rope_append(dq, Hq, cache, (pos if axes > 1 else pos[0]).to(DEV), slot.to(DEV), table.to(DEV) if rot else None,
                      layout=layout, q_norm=w[0].to(DEV) if qn else None, k_norm=w[1].to(DEV) if kn else None, eps=eps,
                      pair_axis=pair_axis if axes > 1 else None)
    torch.cuda.synchronize()
    x = qkv.reshape(M, Hq + 2 * Hkv, D)
    want = F.rotate(x[:, :Hq], w[0], eps, table, pos, listed, layout)
    size = F.rotate(x[:, :Hq].abs(), None if w[0] is None else w[0].abs(), eps, None, pos, listed, layout)
    # as attention_ref.rotate, with both terms of a pair bounded by twice the head's largest normed value
    tol = ((D / 2 if qn else 0) + 12) * R.U32 * 2 * size.amax(-1, keepdim=True)
    R.check(q, want, tol + R.out_roundoff(dtype) * (want.abs() + tol) + 1e-30, "queries")
    k = F.rotate(x[:, Hq:Hq + Hkv], w[1], eps, table, pos, listed, layout).float().double()
    v = x[:, Hq + Hkv:].double()
    for name, y, c, s, (c0, s0) in (("keys", k, cache.k, cache.k_scale, start[0]), ("values", v, cache.v, cache.v_scale, start[1])):
        codes, scale = F.store(c0.double(), s0, y, slots)
        assert torch.equal(s.cpu(), scale), f"{name}: scales"
        F.same(c, codes, name)
    return cache


BATCH = [5, 16 + 15, 64, 96 + 1, 160, 32 + 8, 200, 48]         # single tokens in blocks of their own


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("slots,Hq,Hkv,D,page,layout,rot,qn,kn", [
    ([0], 4, 1, 128, 16, "half", 128, False, False),
    ([7], 32, 8, 128, 16, "half", 128, True, True),
    (BATCH, 6, 2, 128, 16, "half", 64, False, True),
    (BATCH, 5, 5, 64, 32, "interleaved", 64, True, False),
    (list(range(16)), 4, 2, 128, 16, "half", 128, False, True),
    (list(range(50)), 4, 2, 64, 64, "half", 32, True, True),
    (list(range(11, 60)), 8, 1, 128, 32, "interleaved", 128, False, True),      # begins inside a block
    (list(range(3, 25)) + list(range(64, 64 + 33)) + [40] + list(range(130, 143)), 4, 2, 128, 32, "half", 128, True, True),
    (list(range(48, 64)) + list(range(0, 17)), 2, 2, 64, 16, "half", 64, False, False),
    (list(range(32, 48)), 0, 2, 128, 16, "half", 0, False, True),
    # rotated parts that no whole 16-byte chunk holds
    (list(range(5, 27)), 4, 2, 128, 16, "half", 20, True, True),
    (BATCH, 4, 2, 64, 16, "interleaved", 6, False, True),
    (list(range(18)), 4, 2, 128, 16, "half", 2, False, False),
])
def test_append(dtype, slots, Hq, Hkv, D, page, layout, rot, qn, kn):
    run_append(gen(len(slots) + rot), slots, Hq, Hkv, D, page, dtype, layout, rot, qn, kn)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,shift", [(64, 0), (1, 0), (0, 1), (8, 8)])
def test_append_strides(dtype, pad, shift):
    run_append(gen(5), list(range(9, 30)), 4, 2, 128, 16, dtype, "half", 128, True, True, pad=pad, shift=shift)
    run_append(gen(6), BATCH, 4, 2, 64, 16, dtype, "interleaved", 32, False, False, pad=pad, shift=shift)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("axes,kind,layout,rot,D", [
    (3, "blocks", "half", 128, 128), (3, "turns", "half", 64, 64), (2, "turns", "interleaved", 32, 128),
    (4, "blocks", "interleaved", 64, 64), (3, "turns", "half", 22, 64), (3, "blocks", "half", 48, 128)])
def test_append_with_axes(dtype, axes, kind, layout, rot, D):
    run_append(gen(axes), list(range(4, 29)) + BATCH[2:4], 4, 2, D, 16, dtype, layout, rot, True, True, axes=axes, kind=kind)


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("slots", [
    [-1, 0, 1, -1, 18, 19, 99999, 2147483647, 36], [-1] * 40, [9, 3, 4, 40, 33, 32, 47, 20, 22] + list(range(79, 63, -1)), [64] + [-1] * 20 + list(range(16, 40)),
    list(range(80, 112)) + [112, 127]])
def test_append_padding(slots, odd):
    """Rows whose slot is outside the cache store nothing; a block's rows in any order, gaps among them."""
    run_append(gen(9), slots, 4, 2, 128, 16, torch.bfloat16, "half", 128, True, True, pages=8, pad=odd)


def test_append_bad_positions():
    """A position outside the table on any axis: NaN queries, nothing stored."""
    D, Hq, Hkv, M = 128, 2, 1, 6
    g = gen(3)
    qkv = torch.randn(M, (Hq + 2 * Hkv) * D, generator=g).to(torch.bfloat16).to(DEV)
    table = torch.from_numpy(S.rope_table(D, 10)).to(DEV)
    pos = ints([[0, 1, 2, -1, 4, 5], [0, 10, 2, 3, 4, 5]]).to(DEV)
    k, s = random_cache(g, 3, Hkv, 16, D)
    slots = [0, 1, 16, 17, 32, 33]
    for pad in (0, 1):
        cache = S.KvCacheF8(*[c.to(DEV) for c in (k, k, s, s)])
        x = torch.nn.functional.pad(qkv, (0, pad))[:, :qkv.shape[1]]
        q = S.rope_append(x, Hq, cache, pos, ints(slots).to(DEV), table, pair_axis=bytes([0, 1] * 32))
        assert torch.isnan(q[[1, 3]]).all() and not torch.isnan(q[[0, 2, 4, 5]]).any()
        codes, scale = F.store(k.double(), s, qkv.cpu().view(M, -1, D)[:, Hq + Hkv:].double(), [0, -1, 16, -1, 32, 33])
        assert torch.equal(cache.v_scale.cpu(), scale)
        F.same(cache.v, codes)
        kept = [i for i in range(16) if i > 1]
        assert torch.equal(cache.k.cpu().view(torch.uint8)[:, :, kept], k.view(torch.uint8)[:, :, kept])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_special_values(dtype):
    """Zeros, the largest and the smallest numbers, and what is not finite."""
    D, Hkv = 64, 1
    rows = torch.zeros(5, 3 * D, dtype=dtype)
    rows[1, D:] = torch.finfo(dtype).max
    rows[2, D:2 * D] = 1e-37
    rows[2, 2 * D:] = 2.0 ** -126
    rows[3, D:] = torch.linspace(-3, 3, 2 * D).to(dtype)
    rows[3, D + 5], rows[3, D + 6], rows[3, 2 * D + 9] = NAN, INF, -INF
    rows[4, D:] = NAN
    slots = [0, 16, 32, 48, 64]
    start = torch.zeros(6, Hkv, 16, D, dtype=torch.float64), torch.full((6, Hkv, 1), 100, dtype=torch.uint8)
    cache = S.KvCacheF8(*[c.to(DEV) for c in (start[0].to(F.F8), start[0].to(F.F8), start[1], start[1].clone())])
    for pad in (0, 3):
        S.rope_append(torch.nn.functional.pad(rows, (0, pad)).to(DEV)[:, :3 * D], 1, cache, None, ints(slots).to(DEV), None)
        for c, s, y in ((cache.k, cache.k_scale, rows[:, None, D:2 * D]), (cache.v, cache.v_scale, rows[:, None, 2 * D:])):
            codes, scale = F.store(*start, y.double(), slots)
            assert torch.equal(s.cpu(), scale)
            F.same(c, codes)
    assert int(cache.k_scale[0, 0, 0]) == 10 and int(cache.k_scale[1, 0, 0]) == 247


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_token_by_token(dtype):
    """Forty tokens of growing and shrinking size, one call each, and the page used again: scales grow, codes
    are recoded, and the block's first token begins it anew."""
    D, Hkv, Hq, page = 128, 2, 2, 32
    g = gen(11)
    start = random_cache(g, 2, Hkv, page, D)
    cache = S.KvCacheF8(*[c.to(DEV) for c in (start[0], start[0], start[1], start[1].clone())])
    codes, scale = start[0].double(), start[1]
    for t in list(range(40)) + [0, 1, 2, 3]:
        x = (torch.randn(1, (Hq + 2 * Hkv) * D, generator=g) * 2.0 ** ((t * 7) % 13 - 6)).to(dtype)
        S.rope_append(x.to(DEV), Hq, cache, None, ints([t]).to(DEV), None)
        codes, scale = F.store(codes, scale, x.view(1, -1, D)[:, Hq + Hkv:].double(), [t])
        assert torch.equal(cache.v_scale.cpu(), scale), t
        F.same(cache.v, codes, f"token {t}")


def test_append_all_codes_recode():
    """Every code by every power that leaves it something."""
    D = 64
    every = torch.arange(256, dtype=torch.uint8).view(4, 64)
    for d in range(0, 22):
        k = torch.zeros(1, 1, 16, D, dtype=torch.uint8)
        k[0, 0, :4] = every
        s = torch.full((1, 1, 1), 100, dtype=torch.uint8)
        cache = S.KvCacheF8(*[c.to(DEV) for c in (k.view(F.F8), k.view(F.F8), s, s.clone())])
        x = torch.full((1, 3 * D), 448 * 2.0 ** (100 - 127 + d))
        S.rope_append(x.to(DEV), 1, cache, None, ints([4]).to(DEV), None)
        codes, scale = F.store(k.view(F.F8).double(), s, x[:, None, :D].double(), [4])
        assert torch.equal(cache.k_scale.cpu(), scale) and int(scale[0, 0, 0]) == 100 + d
        F.same(cache.k, codes, f"by 2^-{d}")
        # (signs of zeros too)
        neg = cache.k.view(torch.uint8).cpu()[0, 0, :4] >> 7
        assert torch.equal(neg[every != 127], (every >> 7)[every != 127])


def test_append_in_place():
    M, Hq, Hkv, D = 19, 4, 2, 128
    for rot in (128, 20):
        g = gen(2)
        qkv = torch.randn(M, (Hq + 2 * Hkv) * D, generator=g).to(torch.bfloat16).to(DEV)
        table = torch.from_numpy(S.rope_table(rot, 50)).to(DEV)
        pos = torch.arange(M, dtype=torch.int32, device=DEV)
        c = []
        for _ in range(2):
            c.append(S.KvCacheF8.empty(2, Hkv, 16, D))
            for t in (c[-1].k, c[-1].v, c[-1].k_scale, c[-1].v_scale):
                t.view(torch.uint8).zero_()
        apart = S.rope_append(qkv, Hq, c[0], pos, pos, table)
        inside = qkv.clone()
        S.rope_append(inside, Hq, c[1], pos, pos, table, out=inside.view(M, -1, D)[:, :Hq])
        assert torch.equal(inside.view(M, -1, D)[:, :Hq], apart) and torch.equal(inside[:, Hq * D:], qkv[:, Hq * D:])
        for a, b in ((c[0].k, c[1].k), (c[0].v, c[1].v), (c[0].k_scale, c[1].k_scale), (c[0].v_scale, c[1].v_scale)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------ axes onto a cache of the model's own type

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("axes,kind,layout,rot,D,pad,M", [
    (3, "blocks", "half", 128, 128, 0, 1), (3, "turns", "half", 128, 128, 0, 7), (3, "turns", "half", 64, 64, 1, 5),
    (2, "blocks", "interleaved", 32, 128, 0, 9), (4, "turns", "interleaved", 64, 64, 0, 6), (1, "blocks", "half", 48, 64, 0, 3),
    (3, "turns", "interleaved", 22, 64, 0, 4), (3, "blocks", "half", 48, 128, 0, 4200)])
def test_axes(dtype, axes, kind, layout, rot, D, pad, M):
    g = gen(rot + axes)
    Hq, Hkv, page = (4, 2, 16) if M < 100 else (14, 1, 64)
    width = (Hq + 2 * Hkv) * D
    qkv = torch.randn(M, width + pad, generator=g).to(dtype)
    table = torch.from_numpy(S.rope_table(rot, 61, theta=500.0))
    pos = torch.randint(0, 61, (axes, M), generator=g).to(torch.int32)
    pair_axis, listed = axes_of(rot, axes, kind)
    w = 1 + 0.3 * torch.randn(D, generator=g)
    pages = -(-M // page) + 1
    slot = torch.randperm(pages * page, generator=g)[:M].to(torch.int32)
    cache = S.KvCache(*[torch.zeros(pages, Hkv, page, D, dtype=dtype, device=DEV) for _ in range(2)])
    q = S.rope_append(qkv.to(DEV)[:, :width], Hq, cache, pos.to(DEV), slot.to(DEV), table.to(DEV), layout=layout,
                      q_norm=w.to(DEV), k_norm=w.to(DEV), eps=1e-5, pair_axis=listed if M % 2 else pair_axis)
    some = list(range(M)) if M < 100 else [0, 1, 15, 16, 17, M - 2, M - 1]
    x = qkv[some, :width].view(len(some), -1, D)
    for got, y in ((q[some], x[:, :Hq]),
                   (cache.k.transpose(1, 2).reshape(-1, Hkv, D)[slot[some].long().to(DEV)], x[:, Hq:Hq + Hkv])):
        want = F.rotate(y, w, 1e-5, table, pos[:, some], listed, layout)
        size = F.rotate(y.abs(), w.abs(), 1e-5, None, pos, listed, layout)
        tol = (D / 2 + 12) * R.U32 * 2 * size.amax(-1, keepdim=True)
        R.check(got, want, tol + R.out_roundoff(dtype) * (want.abs() + tol) + 1e-30)
    assert torch.equal(cache.v.transpose(1, 2).reshape(-1, Hkv, D)[slot.long().to(DEV)].cpu(), qkv[:, :width].view(M, -1, D)[:, Hq + Hkv:])


def test_one_axis_is_the_plain_call():
    M, Hq, Hkv, D = 40, 4, 2, 128
    g = gen(4)
    qkv = torch.randn(M, (Hq + 2 * Hkv) * D, generator=g).to(torch.bfloat16).to(DEV)
    table = torch.from_numpy(S.rope_table(D, 50)).to(DEV)
    pos = torch.arange(M, dtype=torch.int32, device=DEV)
    got = []
    for kw in (dict(), dict(pair_axis=bytes(64)), dict(pair_axis=[i % 3 for i in range(64)])):
        c = S.KvCache(*[torch.zeros(3, Hkv, 16, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)])
        n = 1 if len(set(kw.get("pair_axis", b"\0"))) == 1 else 3
        p = pos if not kw else pos.expand(n, M).contiguous()
        got.append((S.rope_append(qkv, Hq, c, p, pos, table, **kw), c.k, c.v))
    for a in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(a, got[0]))


# ------------------------------------------------------------------ attention

def filled(g, lens, Hkv, page, D, extra=3):
    """Sequences of these lengths in shuffled pages: codes and scales (CPU), values in 64 bits, the table."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need + [1])), -7, dtype=torch.int32)
    used = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for i in range(need[b]):
            used[table[b, i], :min(page, n - i * page)] = True
    out = []
    for _ in range(2):
        codes = (torch.randn(pages, Hkv, page, D, generator=g) * 100).clamp(-448, 448)
        codes = torch.where(used[:, None, :, None], codes, NAN).to(F.F8)
        scale = torch.randint(118, 121, (pages, Hkv, page // 16), generator=g).to(torch.uint8)
        begun = used.view(pages, -1, 16).any(-1)
        scale = torch.where(begun[:, None], scale, torch.tensor(255, dtype=torch.uint8))
        out += [codes, scale]
    return out[0], out[2], out[1], out[3], table


def run_prefill(seed, new, kv, Hq, Hkv, D, page, dtype, *, scale=None, q_pad=0, o_pad=0):
    g = gen(seed)
    k, v, ks, vs, table = filled(g, kv, Hkv, page, D)
    T = sum(new)
    cu = ints([sum(new[:b]) for b in range(len(new) + 1)])
    row = Hq * D
    base = torch.randn(T * (row + q_pad), generator=g).to(dtype)
    q = torch.as_strided(base, (T, Hq, D), (row + q_pad, D, 1))
    dq = torch.as_strided(base.to(DEV), (T, Hq, D), (row + q_pad, D, 1))
    out = torch.as_strided(torch.full((T * (row + o_pad),), 7.0, dtype=dtype, device=DEV), (T, Hq, D), (row + o_pad, D, 1))
    cache = S.KvCacheF8(*[c.to(DEV) for c in (k, v, ks, vs)])
    got = S.attn_prefill(dq, cu.to(DEV), cache, table.to(DEV), ints(kv).to(DEV), max_len=max(kv), scale=scale, out=out)
    torch.cuda.synchronize()
    want, tol = R.prefill(q, cu, F.values(k, ks), F.values(v, vs), table, kv, D ** -0.5 if scale is None else scale)
    R.check(got, want, tol, f"prefill {new} {kv}")
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,kv,Hq,Hkv,D,page", [
    ([1], [1], 4, 1, 128, 16),
    ([5, 0, 1, 17], [5, 0, 1, 17], 8, 2, 128, 16),
    ([64, 65, 63], [64, 65, 63], 4, 4, 64, 32),
    ([33, 2], [33, 40], 6, 2, 64, 16),
    ([130], [130], 8, 1, 128, 64),
    ([3, 1, 20], [200, 129, 31], 4, 1, 128, 16),
    ([257], [300], 2, 2, 128, 128),
    ([40], [40], 16, 1, 64, 1024),
    ([500, 301], [500, 511], 8, 1, 128, 16),
    ([450], [450], 3, 3, 64, 32),
])
def test_prefill(dtype, new, kv, Hq, Hkv, D, page):
    run_prefill(len(new) * 10 + Hq, new, kv, Hq, Hkv, D, page, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_rows_without_keys(dtype):
    got = run_prefill(3, [10, 6, 40], [4, 0, 5], 4, 2, 128, 16, dtype)
    assert got[:6].count_nonzero() == 0 and got[10:16].count_nonzero() == 0 and got[16:51].count_nonzero() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_strides_and_scale(dtype):
    run_prefill(4, [20, 7], [20, 50], 4, 2, 128, 16, dtype, scale=0.31, q_pad=64, o_pad=8)
    run_prefill(5, [9], [9], 4, 4, 64, 16, dtype, scale=-0.2, q_pad=8, o_pad=24)
    run_prefill(6, [9], [9], 4, 4, 64, 16, dtype, scale=0.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_long_context_in_parts(dtype, D):
    cache = S.KvCacheF8.empty(1, 2, 16, D)
    assert S.attn_prefill_workspace(cache, 3, 26, 4, 2500, dtype=dtype) > 0
    run_prefill(8, [5, 20, 1], [2500, 611, 1024], 4, 2, D, 16, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,old", [(45, 0), (70, 13), (300, 0)])
def test_prefill_what_is_not_seen_has_no_influence(dtype, new, old):
    """A code NaN in the middle of a sequence: the tokens before it come out as without it, bit for bit."""
    Hq, Hkv, D, page, n = 4, 2, 128, 16, new + old
    g = gen(new)
    k, v, ks, vs, table = filled(g, [n], Hkv, page, D)
    q = torch.randn(new, Hq, D, generator=g).to(dtype).to(DEV)
    cu, kv = ints([0, new]).to(DEV), ints([n]).to(DEV)

    def run():
        cache = S.KvCacheF8(*[c.to(DEV) for c in (k, v, ks, vs)])
        return S.attn_prefill(q, cu, cache, table.to(DEV), kv, max_len=n).cpu()

    clean = run()
    for which in (k, v):
        raw = which.view(torch.uint8)
        for at in (old + 21, n - 1):
            p, s = int(table[0, at // page]), at % page
            keep = raw[p, :, s, 5].clone()
            raw[p, :, s, 5] = 0x7F
            got = run()
            raw[p, :, s, 5] = keep
            assert torch.equal(got[:at - old], clean[:at - old])
            if which is v:
                assert not torch.isfinite(got[at - old:, :, 5]).any()
                assert torch.equal(got[..., 6:], clean[..., 6:])
            else:
                assert torch.isnan(got[at - old:]).all()


def run_decode(seed, lens, prefix_len, Hq, Hkv, D, page, dtype, *, scale=None, q_pad=0, o_pad=0, max_len=None):
    g = gen(seed)
    B = len(lens)
    k, v, ks, vs, table = filled(g, lens + [prefix_len], Hkv, page, D)
    prefix, table = table[B, :-(-prefix_len // page)].contiguous(), table[:B].contiguous()
    row = Hq * D
    base = torch.randn(B * (row + q_pad), generator=g).to(dtype)
    q = torch.as_strided(base, (B, Hq, D), (row + q_pad, D, 1))
    dq = torch.as_strided(base.to(DEV), (B, Hq, D), (row + q_pad, D, 1))
    out = torch.as_strided(torch.full((B * (row + o_pad),), 7.0, dtype=dtype, device=DEV), (B, Hq, D), (row + o_pad, D, 1))
    cache = S.KvCacheF8(*[c.to(DEV) for c in (k, v, ks, vs)])
    got = S.attn_decode(dq, cache, table.to(DEV), ints(lens).to(DEV),
                        max_len=max(lens) if max_len is None else max_len, prefix=prefix.to(DEV) if prefix_len else None,
                        prefix_len=prefix_len, scale=scale, out=out)
    torch.cuda.synchronize()
    want, tol = R.decode(q, F.values(k, ks), F.values(v, vs), table, lens, prefix, prefix_len, D ** -0.5 if scale is None else scale)
    R.check(got, want, tol, f"decode {lens} after {prefix_len}")
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,prefix,Hq,Hkv,D,page", [
    ([1], 0, 4, 1, 128, 16),
    ([33], 0, 32, 8, 128, 16),
    ([0, 5, 16, 17], 0, 8, 2, 64, 16),
    ([700, 1, 0, 129], 0, 6, 2, 128, 64),
    ([64, 128], 0, 40, 2, 64, 32),          # 20 query heads to a key/value head
    ([3], 1, 4, 4, 128, 16),
    ([0, 0], 50, 8, 1, 64, 16),
    ([5, 0, 31, 300], 333, 8, 2, 128, 16),
    ([2] * 37, 129, 4, 1, 128, 128),
    ([40, 7, 9], 1500, 12, 4, 64, 16),
    ([9] * 70, 1100, 8, 2, 128, 16),        # 280 rows of the prefix to a key/value head
    ([9] * 70 + [0], 10801, 8, 2, 128, 16),   # enough work for the LDS tiles
    ([3] * 17, 22700, 16, 1, 64, 64),
    ([256, 1, 0, 255], 0, 8, 2, 64, 16),
    ([257, 0, 33, 16], 0, 8, 8, 128, 16),
    ([512, 511, 1], 0, 20, 1, 64, 32),
    ([513, 0, 90], 0, 8, 2, 128, 64),
    ([1, 0, 700, 16, 1024] + [31] * 27, 0, 16, 8, 64, 16),
    ([1025, 0, 300] + [5] * 29, 0, 16, 8, 64, 16),
    ([5000, 4097], 0, 8, 2, 128, 16),
])
def test_decode(dtype, lens, prefix, Hq, Hkv, D, page):
    run_decode(len(lens) + prefix, lens, prefix, Hq, Hkv, D, page, dtype)


@pytest.mark.parametrize("lens,prefix,Hq,Hkv,D,page", [
    ([9] * 70 + [0], 31800, 8, 2, 128, 16),
    ([3] * 17, 22800, 48, 1, 64, 64),
])
def test_decode_after_a_long_prefix_of_codes(lens, prefix, Hq, Hkv, D, page):
    """Enough work that the prefix goes to the tiles also where the cache holds codes."""
    run_decode(7, lens, prefix, Hq, Hkv, D, page, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_strides_scale_and_loose_bound(dtype):
    run_decode(1, [20, 7], 40, 4, 2, 128, 16, dtype, scale=0.3, q_pad=64, o_pad=8)
    run_decode(2, [20, 7], 0, 4, 2, 64, 16, dtype, scale=-0.3, max_len=5000)
    run_decode(3, [20, 0], 17, 4, 2, 64, 16, dtype, max_len=16384)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_without_keys(dtype):
    assert run_decode(1, [0, 0], 0, 4, 2, 128, 16, dtype).count_nonzero() == 0
    assert run_decode(1, [0, 0], 0, 4, 2, 128, 16, dtype, max_len=4000).count_nonzero() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_code_at_every_scale(dtype):
    """One key: the output is the value itself, for all 253 numbers a code stands for and scales over the whole range."""
    D, Hkv = 64, 4
    codes = torch.arange(256, dtype=torch.uint8).view(1, 4, 1, 64).repeat(1, 1, 16, 1)
    codes[codes == 127] = 0
    codes[codes == 255] = 0
    q = torch.zeros(1, Hkv, D, dtype=dtype, device=DEV)
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    for byte in (10, 11, 60, 126, 127, 128, 200, 239):
        s = torch.full((1, Hkv, 1), byte, dtype=torch.uint8)
        cache = S.KvCacheF8(*[c.to(DEV) for c in (codes.view(F.F8), codes.view(F.F8), s, s)])
        want = F.values(codes.view(F.F8), s)[0, :, 0]
        for o in (S.attn_decode(q, cache, one[:, None] * 0, one, max_len=1),
                  S.attn_prefill(q, ints([0, 1]).to(DEV), cache, one[:, None] * 0, one, max_len=1)):
            got = o[0].double().cpu()
            # (fp32's numbers below the normal ones may come out as 0)
            ok = (got == want) | ((want.abs() < 2.0 ** -126) & (got.abs() <= want.abs()))
            assert ok.all(), (byte, got[~ok][:5], want[~ok][:5])


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_then_tokens_equal_one_prompt_of_exact_values(dtype):
    """A prompt stored and attended to, then tokens one by one: each step's output is that of the attention over
    the cache's values as they are then."""
    g = gen(21)
    Hq, Hkv, D, page, n = 4, 2, 128, 16, 37
    table_rope = torch.from_numpy(S.rope_table(D, 64)).to(DEV)
    cache = S.KvCacheF8.empty(5, Hkv, page, D)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.view(torch.uint8).fill_(0x7F)
    pages = ints([[3, 0, 4, 1]])
    width = (Hq + 2 * Hkv) * D

    def slots(a, b):
        return ints([int(pages[0, t // page]) * page + t % page for t in range(a, b)]).to(DEV)

    x = torch.randn(n, width, generator=g).to(dtype).to(DEV)
    pos = torch.arange(64, dtype=torch.int32, device=DEV)
    q = S.rope_append(x, Hq, cache, pos[:n].contiguous(), slots(0, n), table_rope)
    o = S.attn_prefill(q, ints([0, n]).to(DEV), cache, pages.to(DEV), ints([n]).to(DEV), max_len=n)
    values = [F.values(c.cpu(), s.cpu()) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    want, tol = R.prefill(q.cpu(), ints([0, n]), *values, pages, [n], D ** -0.5)
    R.check(o, want, tol, "prompt")
    for t in range(n, 52):
        x = torch.randn(1, width, generator=g).to(dtype).to(DEV) * (1 + t % 3)
        q = S.rope_append(x, Hq, cache, pos[t:t + 1].contiguous(), slots(t, t + 1), table_rope)
        o = S.attn_decode(q, cache, pages.to(DEV), ints([t + 1]).to(DEV), max_len=64)
        values = [F.values(c.cpu(), s.cpu()) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
        want, tol = R.decode(q.cpu(), *values, pages, [t + 1], None, 0, D ** -0.5)
        R.check(o, want, tol, f"token {t}")
