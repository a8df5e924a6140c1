"""serq_rope_append, serq_attn_prefill and serq_attn_decode against plain
64-bit forms (attention_ref.py), at the sizes and masks where they can go
wrong. Unused cache slots hold NaN throughout."""

from __future__ import annotations

import pytest
import torch

import attention_ref as R
import w4a4_linear_layers_amd as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


def rnd(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g).to(dtype)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def filled(g, lens, Hkv, page, D, dtype, extra=3):
    """Sequences of these lengths in shuffled pages of a NaN-filled cache (CPU): k, v, table."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra
    k = torch.full((pages, Hkv, page, D), NAN, dtype=dtype)
    v = torch.full((pages, Hkv, page, D), NAN, dtype=dtype)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need + [1])), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for t in range(0, n, page):
            m = min(page, n - t)
            p = int(table[b, t // page])
            k[p, :, :m] = rnd(g, Hkv, m, D, dtype=dtype)
            v[p, :, :m] = rnd(g, Hkv, m, D, dtype=dtype)
    return k, v, table


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


# ------------------------------------------------------------------ rope_append

def run_append(g, M, Hq, Hkv, D, page, dtype, layout, rot, qn, kn, *, pad=0, shift=0, out_pad=0, eps=1e-5):
    width = (Hq + 2 * Hkv) * D
    flat = rnd(g, M * (width + pad) + shift, dtype=dtype)
    qkv = torch.as_strided(flat, (M, width), (width + pad, 1), shift)
    max_pos = 97
    table = torch.from_numpy(S.rope_table(rot, max_pos, theta=1000.0)) if rot else None
    pos = torch.randint(0, max_pos, (M,), generator=g).to(torch.int32)
    pages = -(-M // page) + 2
    slot = torch.randperm(pages * page, generator=g)[:M].to(torch.int32)
    w = [1 + 0.3 * torch.randn(D, generator=g) if f else None for f in (qn, kn)]
    cache = S.KvCache(torch.full((pages, Hkv, page, D), 3.0, dtype=dtype, device=DEV),
                      torch.full((pages, Hkv, page, D), 5.0, dtype=dtype, device=DEV))
    dflat = flat.to(DEV)
    dq = torch.as_strided(dflat, (M, width), (width + pad, 1), shift)
    out = None
    if out_pad:
        out = torch.as_strided(torch.empty(M * (Hq * D + out_pad), dtype=dtype, device=DEV), (M, Hq, D),
                               (Hq * D + out_pad, D, 1))
    q = S.rope_append(dq, Hq, cache, pos.to(DEV), slot.to(DEV), table.to(DEV) if rot else None, layout=layout,
                      q_norm=w[0].to(DEV) if qn else None, k_norm=w[1].to(DEV) if kn else None, eps=eps, out=out)
    torch.cuda.synchronize()
    x = qkv.reshape(M, Hq + 2 * Hkv, D)
    want, tol = R.rotate(x[:, :Hq], w[0], eps, table, pos, layout, dtype)
    R.check(q, want, tol, "queries")
    wk, tk = R.rotate(x[:, Hq:Hq + Hkv], w[1], eps, table, pos, layout, dtype)
    k, v = cache.k.cpu(), cache.v.cpu()
    stored = torch.zeros(pages * page, dtype=torch.bool)
    for t in range(M):
        s = int(slot[t])
        stored[s] = True
        R.check(k[s // page, :, s % page], wk[t], tk[t], f"key {t}")
        assert torch.equal(v[s // page, :, s % page], x[t, Hq + Hkv:]), f"value {t}"
    rest = ~stored.view(pages, page)
    assert (k.transpose(1, 2)[rest] == 3).all() and (v.transpose(1, 2)[rest] == 5).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,Hq,Hkv,D,page,layout,rot,qn,kn", [
    (1, 4, 1, 128, 16, "half", 128, False, False),
    (1, 32, 8, 128, 16, "half", 128, True, True),
    (3, 5, 5, 64, 32, "interleaved", 64, True, False),
    (7, 6, 2, 128, 16, "half", 64, False, True),
    (5, 6, 3, 64, 64, "half", 16, True, True),
    (4, 8, 1, 64, 16, "interleaved", 16, False, False),
    (4, 2, 2, 128, 16, "half", 0, True, True),
    (33, 24, 8, 64, 16, "half", 64, False, False),
    # rotated parts that no whole 16-byte chunk holds
    (3, 4, 2, 128, 16, "half", 20, True, True),
    (3, 4, 2, 64, 16, "interleaved", 6, False, True),
    (3, 4, 2, 128, 16, "half", 2, False, False),
])
def test_append(dtype, M, Hq, Hkv, D, page, layout, rot, qn, kn):
    run_append(gen(M + rot), M, Hq, Hkv, D, page, dtype, layout, rot, qn, kn)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,shift,out_pad", [(64, 0, 64), (1, 0, 0), (0, 1, 3), (8, 8, 5)])
def test_append_strides(dtype, pad, shift, out_pad):
    run_append(gen(5), 6, 4, 2, 128, 16, dtype, "half", 128, True, True, pad=pad, shift=shift, out_pad=out_pad)
    run_append(gen(6), 6, 4, 2, 64, 16, dtype, "interleaved", 32, False, False, pad=pad, shift=shift, out_pad=out_pad)


@pytest.mark.parametrize("odd", [0, 1])
def test_append_padding_and_bad_positions(odd):
    """Slots outside the cache store nothing; positions outside the table give
    NaN queries and store nothing; the rest is untouched by both. The scalar
    path (odd row stride) alike."""
    M, Hq, Hkv, D, page = 6, 4, 2, 128, 16
    g = gen(1)
    width = (Hq + 2 * Hkv) * D
    qkv = rnd(g, M, width + odd)[:, :width].to(DEV)
    cache = S.KvCache(torch.zeros(2, Hkv, page, D, dtype=torch.bfloat16, device=DEV),
                      torch.zeros(2, Hkv, page, D, dtype=torch.bfloat16, device=DEV))
    table = torch.from_numpy(S.rope_table(D, 10)).to(DEV)
    pos, slot = ints([0, 9, 10, -1, 3, 4]).to(DEV), ints([-1, 31, 2, 3, 32, 2147483647]).to(DEV)
    q = S.rope_append(qkv, Hq, cache, pos, slot, table)
    torch.cuda.synchronize()
    assert torch.isnan(q[2:4]).all() and not torch.isnan(q[[0, 1, 4, 5]]).any()
    want = torch.zeros_like(cache.v)
    want[1, :, 15] = qkv[1].view(-1, D)[Hq + Hkv:]
    assert torch.equal(cache.v, want)
    assert cache.k.count_nonzero() == cache.k[1, :, 15].count_nonzero() > 0


@pytest.mark.parametrize("rot", [128, 20])
def test_append_in_place(rot):
    """The queries may overwrite their own part of the q/k/v rows."""
    M, Hq, Hkv, D = 9, 4, 2, 128
    g = gen(2)
    qkv = rnd(g, M, (Hq + 2 * Hkv) * D).to(DEV)
    table = torch.from_numpy(S.rope_table(rot, 50)).to(DEV)
    pos, slot = torch.arange(M, dtype=torch.int32, device=DEV), torch.arange(M, dtype=torch.int32, device=DEV)
    c = [S.KvCache(torch.zeros(1, Hkv, 16, D, dtype=torch.bfloat16, device=DEV),
                   torch.zeros(1, Hkv, 16, D, dtype=torch.bfloat16, device=DEV)) for _ in range(2)]
    apart = S.rope_append(qkv, Hq, c[0], pos, slot, table)
    inside = qkv.clone()
    S.rope_append(inside, Hq, c[1], pos, slot, table, out=inside.view(M, -1, D)[:, :Hq])
    torch.cuda.synchronize()
    assert torch.equal(inside.view(M, -1, D)[:, :Hq], apart) and torch.equal(inside[:, Hq * D:], qkv[:, Hq * D:])
    assert torch.equal(c[0].k, c[1].k) and torch.equal(c[0].v, c[1].v)


def test_append_special_values_stay_in_their_pair():
    """An infinity reaches its own pair, and values that are not rotated pass
    through bit for bit."""
    D = 128
    qkv = torch.ones(1, 3 * D, dtype=torch.bfloat16, device=DEV)
    qkv[0, 3], qkv[0, 100] = float("inf"), -float("inf")
    cache = S.KvCache(torch.zeros(1, 1, 16, D, dtype=torch.bfloat16, device=DEV),
                      torch.zeros(1, 1, 16, D, dtype=torch.bfloat16, device=DEV))
    table = torch.from_numpy(S.rope_table(64, 8)).to(DEV)
    q = S.rope_append(qkv, 1, cache, ints([5]).to(DEV), ints([0]).to(DEV), table)[0, 0].cpu()
    other = [d for d in range(D) if d not in (3, 35, 100)]
    assert torch.isinf(q[3]) and torch.isinf(q[35]) and q[100] == -float("inf") and torch.isfinite(q[other]).all()


# ------------------------------------------------------------------ prefill

def run_prefill(seed, new, kv, Hq, Hkv, D, page, dtype, *, scale=None, q_pad=0, o_pad=0):
    g = gen(seed)
    k, v, table = filled(g, kv, Hkv, page, D, dtype)
    T = sum(new)
    cu = ints([sum(new[:b]) for b in range(len(new) + 1)])
    row = Hq * D
    base = torch.randn(T * (row + q_pad), generator=g).to(dtype)
    q = torch.as_strided(base, (T, Hq, D), (row + q_pad, D, 1))
    dq = torch.as_strided(base.to(DEV), (T, Hq, D), (row + q_pad, D, 1))
    out = torch.as_strided(torch.full((T * (row + o_pad),), 7.0, dtype=dtype, device=DEV), (T, Hq, D),
                           (row + o_pad, D, 1))
    cache = S.KvCache(k.to(DEV), v.to(DEV))
    got = S.attn_prefill(dq, cu.to(DEV), cache, table.to(DEV), ints(kv).to(DEV), max_len=max(kv), scale=scale, out=out)
    torch.cuda.synchronize()
    want, tol = R.prefill(q, cu, k, v, table, kv, D ** -0.5 if scale is None else scale)
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
    """More new tokens than keys: the first rows see nothing and give zeros;
    a sequence without any key gives zeros throughout."""
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
    """Few new tokens over many keys: the keys are cut in parts and joined."""
    cache = S.KvCache(torch.empty(1, 2, 16, D, dtype=dtype, device=DEV), torch.empty(1, 2, 16, D, dtype=dtype, device=DEV))
    assert S.attn_prefill_workspace(cache, 3, 26, 4, 2500) > 0
    run_prefill(8, [5, 20, 1], [2500, 611, 1024], 4, 2, D, 16, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("what", [NAN, float("inf"), -float("inf")])
@pytest.mark.parametrize("new,old", [(45, 0), (70, 13), (300, 0)])
def test_prefill_what_is_not_seen_has_no_influence(dtype, what, new, old):
    """A key or a value that is not finite, in the middle of a sequence: the
    tokens before it come out as without it, bit for bit."""
    Hq, Hkv, D, page, n = 4, 2, 128, 16, new + old
    g = gen(new)
    k, v, table = filled(g, [n], Hkv, page, D, dtype)
    q = rnd(g, new, Hq, D, dtype=dtype).to(DEV)
    cu, kv = ints([0, new]).to(DEV), ints([n]).to(DEV)

    def run():
        return S.attn_prefill(q, cu, S.KvCache(k.to(DEV), v.to(DEV)), table.to(DEV), kv, max_len=n).cpu()

    clean = run()
    for which in (k, v):
        for at in (old + 21, n - 1):
            p, s = int(table[0, at // page]), at % page
            keep = which[p, :, s, 5].clone()
            which[p, :, s, 5] = what
            got = run()
            which[p, :, s, 5] = keep
            assert torch.equal(got[:at - old], clean[:at - old])
            if which is v:
                assert not torch.isfinite(got[at - old:, :, 5]).any()
                assert torch.equal(got[..., 6:], clean[..., 6:])


# ------------------------------------------------------------------ decode

def run_decode(seed, lens, prefix_len, Hq, Hkv, D, page, dtype, *, scale=None, q_pad=0, o_pad=0, max_len=None):
    g = gen(seed)
    B = len(lens)
    k, v, table = filled(g, lens + [prefix_len], Hkv, page, D, dtype)
    prefix, table = table[B, :-(-prefix_len // page)].contiguous(), table[:B].contiguous()
    row = Hq * D
    base = torch.randn(B * (row + q_pad), generator=g).to(dtype)
    q = torch.as_strided(base, (B, Hq, D), (row + q_pad, D, 1))
    dq = torch.as_strided(base.to(DEV), (B, Hq, D), (row + q_pad, D, 1))
    out = torch.as_strided(torch.full((B * (row + o_pad),), 7.0, dtype=dtype, device=DEV), (B, Hq, D),
                           (row + o_pad, D, 1))
    got = S.attn_decode(dq, S.KvCache(k.to(DEV), v.to(DEV)), table.to(DEV), ints(lens).to(DEV),
                        max_len=max(lens) if max_len is None else max_len, prefix=prefix.to(DEV) if prefix_len else None,
                        prefix_len=prefix_len, scale=scale, out=out)
    torch.cuda.synchronize()
    want, tol = R.decode(q, k, v, table, lens, prefix, prefix_len, D ** -0.5 if scale is None else scale)
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
    ([7] * 33, 600, 8, 1, 64, 32),
    ([9] * 70 + [0], 10801, 8, 2, 128, 16),   # enough work for the LDS tiles
    ([3] * 17, 22700, 16, 1, 64, 64),
])
def test_decode(dtype, lens, prefix, Hq, Hkv, D, page):
    run_decode(len(lens) + prefix, lens, prefix, Hq, Hkv, D, page, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_strides_scale_and_loose_bound(dtype):
    run_decode(1, [20, 7], 40, 4, 2, 128, 16, dtype, scale=0.3, q_pad=64, o_pad=8)
    run_decode(2, [20, 7], 0, 4, 2, 64, 16, dtype, scale=-0.3, max_len=5000)
    run_decode(3, [20, 0], 17, 4, 2, 64, 16, dtype, max_len=16384)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_without_keys(dtype):
    assert run_decode(1, [0, 0], 0, 4, 2, 128, 16, dtype).count_nonzero() == 0
    assert run_decode(1, [0, 0], 0, 4, 2, 128, 16, dtype, max_len=4000).count_nonzero() == 0


# Around the bounds where a sequence's keys are cut in parts or taken whole,
# by four waves or by eight, with few sequences and with many.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [
    ([256, 1, 0, 255], 8, 2, 64, 16),
    ([257, 0, 33, 16], 8, 8, 128, 16),
    ([512, 511, 1], 20, 1, 64, 32),           # two tiles of query heads
    ([513, 0, 90], 8, 2, 128, 64),
    ([1, 0, 700, 16, 1024] + [31] * 27, 16, 8, 64, 16),
    ([1025, 0, 300] + [5] * 29, 16, 8, 64, 16),
])
def test_decode_of_short_caches(dtype, lens, Hq, Hkv, D, page):
    run_decode(7, lens, 0, Hq, Hkv, D, page, dtype)


def test_lengths_beyond_the_bound_are_cut():
    """kv_len above max_len or the table's room counts as that; below 0 as 0."""
    g = gen(9)
    k, v, table = filled(g, [48, 48], 2, 16, 64, torch.bfloat16)
    cache = S.KvCache(k.to(DEV), v.to(DEV))
    q = rnd(g, 2, 4, 64).to(DEV)
    t = table.to(DEV)
    want = S.attn_decode(q, cache, t, ints([30, 0]).to(DEV), max_len=48)
    got = S.attn_decode(q, cache, t, ints([2000000000, -5]).to(DEV), max_len=30)
    assert torch.equal(got, want)
    full = S.attn_decode(q, cache, t, ints([48, 48]).to(DEV), max_len=48)
    loose = S.attn_decode(q, cache, t, ints([49, 2000000000]).to(DEV), max_len=100000)     # the table's room: 48
    assert torch.equal(loose, full)


def test_scores_far_apart():
    """Scores of +-1e4 in base 2: one key takes all, nothing overflows."""
    D, n = 64, 100
    k = torch.zeros(7, 1, 16, D)
    k[:, 0, :, 0] = torch.linspace(-80, 80, 112).view(7, 16)
    v = torch.randn(7, 1, 16, D, generator=gen(0))
    q = torch.zeros(1, 2, D)
    q[0, 0, 0], q[0, 1, 0] = 1000.0, -1000.0
    table = torch.arange(7, dtype=torch.int32)[None].to(DEV)
    for dtype in (torch.float32, torch.bfloat16):
        o = S.attn_decode(q.to(DEV, dtype), S.KvCache(k.to(DEV, dtype), v.to(DEV, dtype)), table, ints([n]).to(DEV),
                          max_len=n, scale=1.0).cpu()
        flat = v.to(dtype).view(-1, D)
        kk = k.to(dtype).double()[..., 0].flatten()[:n]
        for h, sign in ((0, 1), (1, -1)):
            same = kk * sign == (kk * sign).max()
            want = flat[:n][same].double().mean(0)
            assert (o[0, h].double() - want).abs().max() <= (2 ** -8 if dtype == torch.bfloat16 else 2 ** -22) * \
                flat[:n][same].double().abs().max()


def test_offsets_past_32_bits():
    """Pages whose element offsets pass 2^32."""
    D, Hkv, page = 128, 8, 1024
    pages = (1 << 32) // (D * Hkv * page) + 3
    k = torch.empty(pages, Hkv, page, D, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    g = gen(4)
    rows = rnd(g, 40, (8 + 2 * Hkv) * D).to(DEV)
    cache = S.KvCache(k, v)
    small = S.KvCache(torch.zeros(2, Hkv, page, D, dtype=torch.bfloat16, device=DEV),
                      torch.zeros(2, Hkv, page, D, dtype=torch.bfloat16, device=DEV))
    at = torch.arange(40, dtype=torch.int32, device=DEV)
    outs = []
    for c, p in ((cache, pages - 2), (small, 0)):
        q = S.rope_append(rows, 8, c, None, at + p * page, None)
        table = ints([[p, p + 1]]).to(DEV)
        outs.append((S.attn_decode(q[39:], c, table, ints([40]).to(DEV), max_len=40),
                     S.attn_prefill(q, ints([0, 40]).to(DEV), c, table, ints([40]).to(DEV), max_len=40)))
    torch.cuda.synchronize()
    assert torch.equal(cache.k[pages - 2, :, :40], small.k[0, :, :40])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ streams, graphs, workspaces

def _step():
    g = gen(11)
    D, Hq, Hkv, page, B, P = 128, 8, 2, 16, 5, 900
    lens = [3, 0, 40, 600, 17]
    k, v, table = filled(g, lens + [P], Hkv, page, D, torch.bfloat16)
    cache = S.KvCache(k.to(DEV), v.to(DEV))
    prefix, table = table[B, :-(-P // page)].contiguous().to(DEV), table[:B].contiguous().to(DEV)
    q = rnd(g, B, Hq, D).to(DEV)
    cu, new = ints([0, 1, 1, 2, 4, 5]).to(DEV), rnd(g, 5, Hq, D).to(DEV)
    kv = ints(lens).to(DEV)

    def go(out=None):
        a = S.attn_decode(q, cache, table, kv, max_len=4096, prefix=prefix, prefix_len=P, out=out and out[0])
        b = S.attn_prefill(new, cu, cache, table, kv, max_len=4096, out=out and out[1])
        return a, b
    return go


def test_runs_repeat_bit_for_bit_and_on_other_streams():
    go = _step()
    first = go()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = [go() for _ in range(3)]
    side.synchronize()
    for o in other:
        assert torch.equal(o[0], first[0]) and torch.equal(o[1], first[1])


def test_graph_replays():
    """Both calls with their joins in a captured graph, replayed with eager
    work in between, each replay against the eager result."""
    go = _step()
    want = go()
    torch.cuda.synchronize()
    outs = [torch.empty_like(x) for x in want]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        go(outs)
    side.synchronize()
    with torch.cuda.graph(graph):
        go(outs)
    for _ in range(4):
        for o in outs:
            o.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
        again = go()
        torch.cuda.synchronize()
        assert torch.equal(again[0], want[0])


def test_dirty_workspace_does_not_matter():
    g = gen(12)
    k, v, table = filled(g, [900, 30], 2, 16, 64, torch.bfloat16)
    cache = S.KvCache(k.to(DEV), v.to(DEV))
    q = rnd(g, 2, 8, 64).to(DEV)
    need = S.attn_decode_workspace(cache, 2, 8, 0, 900)
    assert need > 0
    outs = []
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        outs.append(S.attn_decode(q, cache, table.to(DEV), ints([900, 30]).to(DEV), max_len=900, workspace=ws))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])


def test_prefill_in_place():
    """O may be Q."""
    g = gen(13)
    k, v, table = filled(g, [70, 1500], 2, 16, 128, torch.bfloat16)
    cache = S.KvCache(k.to(DEV), v.to(DEV))
    q = rnd(g, 90, 8, 128).to(DEV)
    args = (ints([0, 70, 90]).to(DEV), cache, table.to(DEV), ints([70, 1500]).to(DEV))
    apart = S.attn_prefill(q, *args, max_len=1500)
    S.attn_prefill(q, *args, max_len=1500, out=q)
    torch.cuda.synchronize()
    assert torch.equal(q, apart)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefill_many_sequences(dtype):
    """More sequences than a wave has lanes, and as many as it has: empty
    ones, equal lengths, old contexts among them."""
    new = [(7 * i) % 5 for i in range(130)]
    kv = [n + (11 * i) % 23 if n else (i % 3) for i, n in enumerate(new)]
    run_prefill(21, new, kv, 2, 1, 64, 16, dtype)
    run_prefill(22, new[:64], kv[:64], 2, 1, 64, 16, dtype)
    run_prefill(23, [70, 0, 70, 1, 33, 70], [70, 9, 75, 300, 33, 70], 2, 2, 64, 16, dtype)
