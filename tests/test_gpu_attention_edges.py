"""The attention calls at the edges of their arguments and in the kernels that
only large calls reach, against 64-bit forms (attention_ref.py)."""

from __future__ import annotations

import pytest
import torch

import attention_ref as R
import w4a4_linear_layers_amd as S
from test_gpu_attention import DEV, filled, gen, ints, rnd

pytestmark = pytest.mark.gpu
TYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


# ------------------------------------------------------------------ scales

@TYPES
@pytest.mark.parametrize("scale,size", [(0.0, 1e15), (-0.0, 1.0), (1e-32, 1e16), (-1e-32, 1e16), (1e-37, 1.5e18),
                                        (5e-39, 1.5e18)])
def test_scores_of_any_size_under_a_scale_to_match(dtype, scale, size):
    """Products of queries and keys far above what a small scale makes of
    them; scale 0 weighs all keys alike. Prompt, own tokens and a prefix of
    enough work for the LDS tiles (bf16)."""
    Hq, Hkv, D, page = 8, 1, 64, 16
    g = gen(31)
    new, kv = [70, 1, 5], [70, 300, 5]
    k, v, table = filled(g, kv, Hkv, page, D, dtype)
    k = (k.float() * size).to(dtype)
    q = (rnd(g, sum(new), Hq, D, dtype=torch.float32) * size).to(dtype)
    cu = ints([0, 70, 71, 76])
    cache = S.KvCache(k.to(DEV), v.to(DEV))
    got = S.attn_prefill(q.to(DEV), cu.to(DEV), cache, table.to(DEV), ints(kv).to(DEV), max_len=300, scale=scale)
    R.check(got, *R.prefill(q, cu, k, v, table, kv, scale), f"prefill, scale {scale}")

    lens, P = [40, 0, 3] * 6, 42000                       # 18 x 8 x 42000 = 6.05 million
    k, v, table = filled(g, lens + [P], Hkv, page, D, dtype)
    k = (k.float() * size).to(dtype)
    prefix, table = table[len(lens)], table[:len(lens), :3].contiguous()
    q = (rnd(g, len(lens), Hq, D, dtype=torch.float32) * size).to(dtype)
    cache = S.KvCache(k.to(DEV), v.to(DEV))
    got = S.attn_decode(q.to(DEV), cache, table.to(DEV), ints(lens).to(DEV), max_len=40, scale=scale,
                        prefix=prefix.to(DEV), prefix_len=P)
    R.check(got, *R.decode(q, k, v, table, lens, prefix, P, scale), f"prefix, scale {scale}")
    got = S.attn_decode(q.to(DEV), cache, table.to(DEV), ints(lens).to(DEV), max_len=40, scale=scale)
    R.check(got, *R.decode(q, k, v, table, lens, None, 0, scale), f"decode, scale {scale}")


# ------------------------------------------------------------------ scores of -inf

@TYPES
@pytest.mark.parametrize("what", [float("inf"), -float("inf"), float("nan")])
def test_rows_whose_scores_are_all_minus_infinity(dtype, what):
    """They give zeros, whatever their values hold; other rows come out as
    they do by themselves."""
    Hq, Hkv, D, page = 8, 2, 128, 16
    g = gen(32)
    new, kv = [40, 33, 3], [40, 90, 2000]
    k, v, table = filled(g, kv, Hkv, page, D, dtype)
    q = rnd(g, sum(new), Hq, D, dtype=dtype)
    q[40:73, :, 7] = 1.0                                   # the second sequence's scores are -inf throughout
    dead = table[1, :6].long()
    k[dead, :, :, 7] = -float("inf")
    v[dead, :, 3, 9] = what

    def prefill():
        return S.attn_prefill(q.to(DEV), ints([0, 40, 73, 76]).to(DEV), S.KvCache(k.to(DEV), v.to(DEV)), table.to(DEV),
                              ints(kv).to(DEV), max_len=2000).cpu()

    def decode(max_len, prefix, prefix_len):
        return S.attn_decode(torch.stack([q[0], q[40], q[73]]).to(DEV), S.KvCache(k.to(DEV), v.to(DEV)),
                             table.to(DEV), ints([40, 90, 500]).to(DEV), max_len=max_len, prefix=prefix,
                             prefix_len=prefix_len).cpu()

    runs = [prefill, lambda: decode(500, None, 0), lambda: decode(2000, None, 0)]
    got = [f() for f in runs]
    v[dead, :, 3, 9] = 0.0
    for a, f in zip(got, runs):
        b = f()
        at = slice(40, 73) if a.shape[0] == 76 else slice(1, 2)
        assert a[at].count_nonzero() == 0 and torch.equal(a, b)

    # a prefix of such scores, and nothing after it, by rows and (bf16) by tiles
    B, P = 20, 40000                                       # 20 x 8 x 40000 = 6.4 million
    for n in (90, P):
        k, v, table = filled(g, [n], Hkv, page, D, dtype)
        k[..., 7] = -float("inf")
        v[..., 5, 9] = what
        q = rnd(g, B, Hq, D, dtype=dtype)
        q[..., 7] = 1.0
        o = S.attn_decode(q.to(DEV), S.KvCache(k.to(DEV), v.to(DEV)), torch.zeros(B, 1, dtype=torch.int32, device=DEV),
                          ints([0] * B).to(DEV), max_len=0, prefix=table[0].to(DEV), prefix_len=n)
        assert o.count_nonzero() == 0


# ------------------------------------------------------------------ norms of tiny heads

@TYPES
@pytest.mark.parametrize("layout,rot", [("half", 128), ("half", 20)])
def test_norms_of_heads_whose_mean_square_is_denormal(dtype, layout, rot):
    """Values of about 2^-64 and eps 0: the mean square is below the normal
    numbers of fp32. A square is then off by 2^-150 at most, D of them by 2^-22
    of their sum, and so is the mean: 2^-21 more of the result at most."""
    M, Hq, Hkv, D, page = 5, 4, 2, 128, 16
    g = gen(33)
    x = (torch.randn(M, Hq + 2 * Hkv, D, generator=g) * 2.0 ** -64).to(dtype)
    w = [1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)]
    table = torch.from_numpy(S.rope_table(rot, 9))
    pos = ints([0, 8, 3, 5, 1])
    cache = S.KvCache.empty(1, Hkv, page, D, dtype=dtype)
    q = S.rope_append(x.view(M, -1).to(DEV), Hq, cache, pos.to(DEV), ints(range(M)).to(DEV), table.to(DEV),
                      layout=layout, q_norm=w[0].to(DEV), k_norm=w[1].to(DEV), eps=0.0)
    for got, part, n in ((q, x[:, :Hq], 0), (cache.k[0, :, :M].transpose(0, 1), x[:, Hq:Hq + Hkv], 1)):
        want, tol = R.rotate(part, w[n], 0.0, table, pos, layout, dtype)
        size, _ = R.rotate(part.abs(), w[n].abs(), 0.0, table.abs(), pos, layout, dtype)
        R.check(got, want, tol + 2.0 ** -21 * size.abs().max(), "norm")


# ------------------------------------------------------------------ calls of more than one launch

def test_append_of_more_tokens_than_a_launch_takes():
    """2^24 + 3 tokens: the last ones, a few in the middle and the first are
    stored, the rest are padding."""
    M, D, page = (1 << 24) + 3, 64, 16
    qkv = torch.zeros(M, 2 * D, dtype=torch.bfloat16, device=DEV)
    at = [0, 5, (1 << 23) - 1, 1 << 23, (1 << 24) - 1, 1 << 24, M - 1]
    rows = rnd(gen(34), len(at), 2 * D).to(DEV)
    qkv[at] = rows
    slot = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    slot[at] = torch.arange(len(at), dtype=torch.int32, device=DEV)
    pos = torch.full((M,), 3, dtype=torch.int32, device=DEV)
    pos[at] = torch.arange(len(at), dtype=torch.int32, device=DEV)
    table = torch.from_numpy(S.rope_table(D, 9)).to(DEV)
    big, small = (S.KvCache(torch.zeros(1, 1, page, D, dtype=torch.bfloat16, device=DEV),
                            torch.zeros(1, 1, page, D, dtype=torch.bfloat16, device=DEV)) for _ in range(2))
    S.rope_append(qkv, 0, big, pos, slot, table)
    S.rope_append(rows, 0, small, pos[at].contiguous(), slot[at].contiguous(), table)
    assert torch.equal(big.k, small.k) and torch.equal(big.v, small.v) and small.k.count_nonzero() > 0


@pytest.mark.parametrize("prefix_len", [0, 40])
def test_decode_of_more_sequences_than_a_launch_takes(prefix_len):
    """2^23 + 5 sequences, most of them without tokens of their own: with a
    prefix every one gives what a call for it alone does."""
    B, Hq, D, page = (1 << 23) + 5, 1, 64, 16
    g = gen(35)
    cache = S.KvCache(rnd(g, 24, 1, page, D).to(DEV), rnd(g, 24, 1, page, D).to(DEV))
    at = [0, 1, (1 << 22) - 1, 1 << 22, (1 << 23) - 1, 1 << 23, B - 1]
    q = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    q[at] = rnd(g, len(at), Hq, D).to(DEV)
    kv = torch.zeros(B, dtype=torch.int32, device=DEV)
    kv[at] = ints([3, 17, 300, 40, 299, 1, 100]).to(DEV)
    table = torch.zeros(B, 19, dtype=torch.int32, device=DEV)
    table[at] = torch.stack([torch.randperm(21, generator=g)[:19].to(torch.int32) for _ in at]).to(DEV)
    prefix = ints([21, 22, 23]).to(DEV) if prefix_len else None
    call = dict(max_len=300, prefix=prefix, prefix_len=prefix_len)
    o = S.attn_decode(q, cache, table, kv, **call)
    for i in at:
        one = S.attn_decode(q[i:i + 1], cache, table[i:i + 1], kv[i:i + 1], **call)
        # (parts of the keys are cut otherwise there: two roundings of the same sum)
        assert (o[i].float() - one[0].float()).abs().max() <= 2.0 ** -7 * cache.v.float().abs().max()
    rest = torch.ones(B, dtype=torch.bool, device=DEV)
    rest[at] = False
    if prefix_len:
        own = cache.v[21:24].reshape(-1, D)[:prefix_len].double().mean(0).to(torch.bfloat16)
        assert (o[:, 0][rest].float() - own.float()).abs().max() <= 2.0 ** -7 * cache.v.float().abs().max()
    else:
        assert o[rest].count_nonzero() == 0


# ------------------------------------------------------------------ kernels that large calls alone reach

def attend64(q, k, v, seen, scale, dtype):
    """q: rows x D of one key/value head, k, v: n x D in 64 bits; row i sees
    the first seen[i] keys. (output, tolerance), the bounds of attention_ref."""
    n, D = k.shape
    q = q.double()
    if n == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    gone = torch.arange(n) >= seen[:, None]
    z = (q @ k.t().contiguous() * scale).masked_fill(gone, -float("inf"))
    p = torch.exp(z - z.amax(1, keepdim=True).clamp(min=-1e300))
    p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    e_z = (q.abs() @ k.abs().t().contiguous()).masked_fill(gone, 0.0).amax(1, keepdim=True)
    e_z = e_z * ((D + 4) * R.U32 * abs(scale))
    o, A = p @ v, p @ v.abs()
    tol = A * 2 * (e_z + (seen[:, None] / 8 + 64) * R.U32) + (A * R.UBF if dtype == torch.bfloat16 else 0)
    return o, tol + R.out_roundoff(dtype) * (o.abs() + tol) + 1e-30


def decode64(q, k, v, table, lens, prefix, P, scale):
    B, Hq, D = q.shape
    G = Hq // k.shape[1]
    o, tol = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    for h in range(k.shape[1]):
        lead = [R.sequence(c, prefix, P, h) for c in (k, v)] if P else [torch.zeros(0, D, dtype=torch.float64)] * 2
        for b, n in enumerate(lens):
            ks, vs = (torch.cat([a, R.sequence(c, table[b], n, h)]) for a, c in zip(lead, (k, v)))
            o[b, h * G:h * G + G], tol[b, h * G:h * G + G] = attend64(q[b, h * G:h * G + G], ks, vs,
                                                                      torch.full((G,), P + n), scale, q.dtype)
    return o, tol


def prefill64(q, cu, k, v, table, kv, scale):
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    o, tol = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    for b, n in enumerate(kv):
        q0, q1 = int(cu[b]), int(cu[b + 1])
        seen = (n - (q1 - q0) + 1 + torch.arange(q1 - q0)).clamp(min=0)
        for h in range(k.shape[1]):
            ks, vs = (R.sequence(c, table[b], n, h) for c in (k, v))
            for j in range(h * G, h * G + G):
                o[q0:q1, j], tol[q0:q1, j] = attend64(q[q0:q1, j], ks, vs, seen, scale, q.dtype)
    return o, tol


def spoiled(need):
    """A workspace of NaN."""
    return torch.full((need,), 255, dtype=torch.uint8, device=DEV) if need else None


@TYPES
@pytest.mark.parametrize("lens,prefix,Hq,Hkv,D", [
    # 2079 rows (not a multiple of the join's four) of 63 parts, and 8 or more of a prefix
    ([8064, 0, 130] + [5, 0, 70] * 10, 1000, 63, 1, 64),
    ([8064, 129, 0] + [128, 1, 300] * 10, 0, 63, 1, 128),
    # a prefix of enough work for the LDS tiles (bf16), 3000 rows of it
    ([40, 0, 300] * 25, 2100, 40, 2, 128),
    ([1, 700, 0] * 13 + [2], 2700, 64, 1, 64),
])
def test_decode_with_many_rows_to_join(dtype, lens, prefix, Hq, Hkv, D):
    g, B, page = gen(41), len(lens), 16
    k, v, table = filled(g, lens + [prefix], Hkv, page, D, dtype)
    lead, table = table[B, :-(-prefix // page)].contiguous(), table[:B].contiguous()
    q = rnd(g, B, Hq, D, dtype=dtype)
    cache = S.KvCache(k.to(DEV), v.to(DEV))
    need = S.attn_decode_workspace(cache, B, Hq, prefix, max(lens))
    assert B * Hq > 2048 and need > 0
    got = S.attn_decode(q.to(DEV), cache, table.to(DEV), ints(lens).to(DEV), max_len=max(lens),
                        prefix=lead.to(DEV) if prefix else None, prefix_len=prefix, workspace=spoiled(need))
    R.check(got, *decode64(q, k, v, table, lens, lead, prefix, D ** -0.5), "decode")


@TYPES
@pytest.mark.parametrize("new,kv,Hq,Hkv,D,in_place", [
    # more than 2048 rows really cut in parts, joined by a wave each: 8 heads to
    # a workgroup (bf16), and 2107 rows of heads that share no workgroup
    ([101, 99, 101], [3000, 700, 1500], 8, 1, 128, False),
    ([150, 0, 151], [2600, 4, 151], 7, 1, 64, True),
    # one token each of sequences over long contexts: fewer parts than the
    # host's bound foresaw, on either side of 64 sequences ...
    ([1] * 40, [8000, 3, 0, 500] * 10, 8, 1, 64, True),
    ([1] * 70, [2600, 64, 65, 1, 1300] * 14, 4, 1, 128, False),
    # ... and one part alone, which is then the output
    ([1] * 40, [2500, 3, 0, 500] * 10, 32, 8, 64, True),
    ([1] * 300, [2500, 3, 0, 500, 1, 7] * 50, 8, 1, 64, False),
])
def test_prefill_in_parts_of_the_device_s_count(dtype, new, kv, Hq, Hkv, D, in_place):
    g, page, T = gen(42), 16, sum(new)
    k, v, table = filled(g, kv, Hkv, page, D, dtype)
    cu = ints([sum(new[:b]) for b in range(len(new) + 1)])
    q = rnd(g, T, Hq, D, dtype=dtype)
    cache, dq = S.KvCache(k.to(DEV), v.to(DEV)), q.to(DEV)
    need = S.attn_prefill_workspace(cache, len(new), T, Hq, max(kv))
    assert need > 0
    got = S.attn_prefill(dq, cu.to(DEV), cache, table.to(DEV), ints(kv).to(DEV), max_len=max(kv),
                         out=dq if in_place else None, workspace=spoiled(need))
    R.check(got, *prefill64(q, cu, k, v, table, kv, D ** -0.5), "prefill")


def rotate64(x, w, eps, table, pos, layout, dtype):
    """attention_ref.rotate for many tokens at once."""
    M, H, D = x.shape
    x, slack = x.double(), 12.0
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
        slack += D / 2
    rot = table.shape[1]
    c, s = (t.double()[:, None] for t in table[pos.long()].split(rot // 2, 1))
    at = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., at[0]], x[..., at[1]]
    y, size = x.clone(), x.abs()
    y[..., at[0]], y[..., at[1]] = a * c - b * s, b * c + a * s
    size[..., at[0]], size[..., at[1]] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    tol = slack * R.U32 * size
    return y, tol + R.out_roundoff(dtype) * (y.abs() + tol) + 1e-30


@TYPES
@pytest.mark.parametrize("Hq,Hkv,D,layout,rot,qn,kn,in_place", [
    (32, 8, 128, "half", 128, True, True, False),       # three whole sets of heads (bf16)
    (33, 11, 128, "interleaved", 64, True, False, True),      # sets that no three divide, a last one in part
    (30, 5, 64, "half", 64, False, True, True),
    (55, 5, 64, "interleaved", 16, True, True, False),
])
def test_append_of_many_normed_tokens(dtype, Hq, Hkv, D, layout, rot, qn, kn, in_place):
    """From 4096 normed tokens a lane has several heads: against the formula,
    and bit for bit against the same tokens in smaller calls."""
    M, page, eps = 4099, 16, 1e-5
    g = gen(43)
    x = rnd(g, M, Hq + 2 * Hkv, D, dtype=dtype)
    w = [1 + 0.3 * torch.randn(D, generator=g) if f else None for f in (qn, kn)]
    table = torch.from_numpy(S.rope_table(rot, 512, theta=1000.0))
    pos = torch.randint(0, 512, (M,), generator=g).to(torch.int32)
    pages = -(-M // page) + 1
    slot = torch.randperm(pages * page, generator=g)[:M].to(torch.int32)
    slot[77] = -1
    outs = []
    for step in (M, 2000):
        cache = S.KvCache(*(torch.zeros(pages, Hkv, page, D, dtype=dtype, device=DEV) for _ in range(2)))
        rows = x.to(DEV).view(M, -1)
        q = rows.view(M, -1, D)[:, :Hq] if in_place else torch.empty(M, Hq, D, dtype=dtype, device=DEV)
        for t in range(0, M, step):
            e = slice(t, t + step)
            S.rope_append(rows[e], Hq, cache, pos[e].to(DEV), slot[e].to(DEV), table.to(DEV), layout=layout,
                          q_norm=w[0].to(DEV) if qn else None, k_norm=w[1].to(DEV) if kn else None, eps=eps, out=q[e])
        assert torch.equal(rows.view(M, -1, D)[:, Hq:].cpu(), x[:, Hq:])
        outs.append((q.cpu(), cache.k.cpu(), cache.v.cpu()))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    q, k, v = outs[0]
    R.check(q, *rotate64(x[:, :Hq], w[0], eps, table, pos, layout, dtype), "queries")
    kept = slot >= 0
    flat_k, flat_v = (c.transpose(1, 2).reshape(-1, Hkv, D) for c in (k, v))
    want, tol = rotate64(x[:, Hq:Hq + Hkv], w[1], eps, table, pos, layout, dtype)
    R.check(flat_k[slot[kept].long()], want[kept], tol[kept], "keys")
    assert torch.equal(flat_v[slot[kept].long()], x[kept][:, Hq + Hkv:])
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[slot[kept].long()] = False
    assert flat_k[rest].count_nonzero() == 0 and flat_v[rest].count_nonzero() == 0
