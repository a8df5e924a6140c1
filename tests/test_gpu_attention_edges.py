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
    q = S.rope_append(x.view(M, -1).to(DEV), Hq, cache, pos.to(DEV), ints(range(M)).to(DEV), table.to(DEV), layout=layout,
                      q_norm=w[0].to(DEV), k_norm=w[1].to(DEV), eps=0.0)
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
