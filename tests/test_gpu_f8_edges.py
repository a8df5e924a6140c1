"""The cache in 8 bits and the linear in 8-bit integers at the edges of their
arguments: far pages, calls of more than one launch, many tokens in runs that
cross every window, streams, the values of the bound."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as R
import f8_ref as F
import w4a4_linear_layers_amd as S
from test_gpu_f8_cache import DEV, NAN, INF, filled, gen, ints, random_cache

pytestmark = pytest.mark.gpu
TYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


def rotate_all(x, w, eps, table, pos):
    """f8_ref.rotate for one axis and half layout, all rows at once."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    if table is None:
        return x
    t = table.double()[pos.long()][:, None]
    h = t.shape[-1] // 2
    c, s = t[..., :h], t[..., h:]
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., 2 * h:]], -1)


@TYPES
@pytest.mark.parametrize("M,Hkv,D,rot,norm,lead", [(4096, 2, 128, 128, True, 0), (4211, 3, 64, 64, True, 5), (5003, 5, 128, 64, False, 9),
                                                   (4100, 1, 64, 0, True, 15), (2500, 2, 128, 128, True, 11),
                                                   (2047, 3, 128, 64, True, 6), (2048, 3, 64, 64, False, 2)])
def test_append_of_many_tokens(dtype, M, Hkv, D, rot, norm, lead):
    """Prompts one after another, each in pages of its own, that begin `lead` tokens inside a block they share with
    earlier ones, so that runs cross windows in every way; some end with a row of padding."""
    g = gen(M)
    Hq, page = 2 * Hkv, 32
    lens, left = [], M
    while left:
        n = min(left, int(torch.randint(1, 400, (1,), generator=g)))
        lens.append(n)
        left -= n
    slot, at = [], 0
    for i, n in enumerate(lens):
        slot += range(at + lead, at + lead + n)
        at += -(-(n + lead) // page) * page
        if i % 4 == 1:
            slot[-1] = -1
    pages = at // page
    qkv = torch.randn(M, (Hq + 2 * Hkv) * D, generator=g).to(dtype)
    table = torch.from_numpy(S.rope_table(rot, 300, theta=900.0)) if rot else None
    pos = torch.randint(0, 300, (M,), generator=g).to(torch.int32)
    w = 1 + 0.3 * torch.randn(D, generator=g) if norm else None
    k, s = random_cache(g, pages, Hkv, page, D)
    cache = S.KvCacheF8(*[c.to(DEV) for c in (k, k, s, s.clone())])
    eps = float(np.float32(1e-6))
    dw = w.to(DEV) if norm else None
    q = S.rope_append(qkv.to(DEV), Hq, cache, pos.to(DEV), ints(slot).to(DEV), table.to(DEV) if rot else None, q_norm=dw,
                      k_norm=dw, eps=eps)
    x = qkv.view(M, -1, D)
    y = rotate_all(x[:, Hq:Hq + Hkv], w, eps, table, pos).float().double()
    for name, y, c, cs in (("keys", y, cache.k, cache.k_scale), ("values", x[:, Hq + Hkv:].double(), cache.v, cache.v_scale)):
        codes, scale = F.store(k.double(), s, y, slot)
        assert int((cs.cpu() != scale).sum()) == 0, name
        F.same(c, codes, name)
    plain = S.KvCache(*[torch.zeros(pages, Hkv, page, D, dtype=dtype, device=DEV) for _ in range(2)])
    again = S.rope_append(qkv.to(DEV), Hq, plain, pos.to(DEV), ints(slot).to(DEV), table.to(DEV) if rot else None, q_norm=dw,
                          k_norm=dw, eps=eps)
    assert torch.equal(q, again)                 # the queries are those of a cache of the model's type


def test_append_of_more_heads_than_a_launch_takes():
    """8190 tokens of 8192 heads of each kind: two launches, with a run across them."""
    M, H, D = 8190, 8192, 64
    at = [0, 5] + list(range(8165, 8186)) + [8189]
    slots = [17, 33] + list(range(64 + 3, 64 + 24)) + [100]
    qkv = torch.zeros(M, 3 * H * D, dtype=torch.bfloat16, device=DEV)
    rows = torch.randn(len(at), 3 * H * D, device=DEV, generator=torch.Generator(DEV).manual_seed(3)).to(torch.bfloat16)
    qkv[at] = rows
    slot = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    slot[at] = ints(slots).to(DEV)
    pos = torch.full((M,), 1, dtype=torch.int32, device=DEV)
    table = torch.from_numpy(S.rope_table(D, 9)).to(DEV)
    caches = []
    for _ in range(2):
        c = S.KvCacheF8.empty(8, H, 16, D)
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            t.view(torch.uint8).fill_(100)
        caches.append(c)
    q = S.rope_append(qkv, H, caches[0], pos, slot, table)
    small = S.rope_append(rows, H, caches[1], pos[:len(at)].contiguous(), ints(slots).to(DEV), table)
    assert torch.equal(q[at], small) and small.count_nonzero() > 0
    a, b = caches
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert (a.k_scale[4] != 100).all()


@TYPES
def test_pages_beyond_4_gb(dtype):
    """Stored to and read from pages whose byte offsets pass 32 bits."""
    D, Hkv, Hq, page, n = 128, 8, 16, 16, 45
    pages = (1 << 32) // (Hkv * page * D) + 9
    cache = S.KvCacheF8.empty(pages, Hkv, page, D)
    ids = [pages - 1, pages - 7, 3]
    for i in ids:
        for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
            t[i].view(torch.uint8).fill_(0x7F)
    g = gen(8)
    slot = [ids[t // page] * page + t % page for t in range(n)]
    qkv = torch.randn(n, (Hq + 2 * Hkv) * D, generator=g).to(dtype)
    q = S.rope_append(qkv.to(DEV), Hq, cache, None, ints(slot).to(DEV), None)
    table, kv = ints([ids]).to(DEV), ints([n]).to(DEV)
    x = qkv.view(n, -1, D)
    zero = torch.full((3, Hkv, page, D), NAN, dtype=torch.float64), torch.full((3, Hkv, 1), 0x7F, dtype=torch.uint8)
    values = []
    for y, c, s in ((x[:, Hq:Hq + Hkv], cache.k, cache.k_scale), (x[:, Hq + Hkv:], cache.v, cache.v_scale)):
        codes, scale = F.store(*zero, y.double(), list(range(n)))
        assert torch.equal(s[ids].cpu(), scale)
        F.same(c.view(torch.uint8)[ids].view(F.F8), codes)
        values.append(F.values(codes, scale))
    o = S.attn_prefill(q, ints([0, n]).to(DEV), cache, table, kv, max_len=n)
    R.check(o, *R.prefill(q.cpu(), ints([0, n]), *values, ints([[0, 1, 2]]), [n], D ** -0.5))
    o = S.attn_decode(q[-1:], cache, table, kv, max_len=n)
    R.check(o, *R.decode(q[-1:].cpu(), *values, ints([[0, 1, 2]]), [n], None, 0, D ** -0.5))


@TYPES
def test_two_streams_at_once(dtype):
    """Calls on two streams, each with a workspace of its own, and tensors made on another stream."""
    g = gen(12)
    lens, Hq, Hkv, D, page = [3000, 41, 900], 16, 4, 128, 16
    k, v, ks, vs, table = filled(g, lens, Hkv, page, D)
    cache = S.KvCacheF8(*[c.to(DEV) for c in (k, v, ks, vs)])
    q = torch.randn(3, Hq, D, generator=g).to(dtype).to(DEV)
    table, kv = table.to(DEV), ints(lens).to(DEV)
    want = S.attn_decode(q, cache, table, kv, max_len=3000)
    cu = ints([0, 1, 2, 3]).to(DEV)
    want2 = S.attn_prefill(q, cu, cache, table, kv, max_len=3000)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(S.attn_decode_workspace(cache, 3, Hq, 0, 3000, dtype=dtype), dtype=torch.uint8, device=DEV),
              torch.empty(max(1, S.attn_prefill_workspace(cache, 3, 3, Hq, 3000, dtype=dtype)), dtype=torch.uint8, device=DEV)]
    got = [[], []]
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            got[0].append(S.attn_decode(q, cache, table, kv, max_len=3000, workspace=spaces[0]))
        with torch.cuda.stream(streams[1]):
            got[1].append(S.attn_prefill(q, cu, cache, table, kv, max_len=3000, workspace=spaces[1]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got[0]) and all(torch.equal(o, want2) for o in got[1])


@TYPES
@pytest.mark.parametrize("what", [INF, -INF, NAN])
def test_queries_that_are_not_finite(dtype, what):
    """Each row stays by itself: the others come out as without it."""
    g = gen(14)
    lens, Hq, Hkv, D, page = [70, 33], 8, 2, 64, 16
    k, v, ks, vs, table = filled(g, lens, Hkv, page, D)
    cache = S.KvCacheF8(*[c.to(DEV) for c in (k, v, ks, vs)])
    q = torch.randn(103, Hq, D, generator=g).to(dtype).to(DEV)
    cu, kv, table = ints([0, 70, 103]).to(DEV), ints(lens).to(DEV), table.to(DEV)
    clean = S.attn_prefill(q, cu, cache, table, kv, max_len=70)
    q[20, 3] = what
    got = S.attn_prefill(q, cu, cache, table, kv, max_len=70)
    rest = torch.ones(103, Hq, dtype=torch.bool, device=DEV)
    rest[20, 3] = False
    assert torch.equal(got[rest], clean[rest])
    one = S.attn_decode(q[19:21], cache, table, kv, max_len=70)
    q[20, 3] = 1.0
    ok = S.attn_decode(q[19:21], cache, table, kv, max_len=70)
    rest = torch.ones(2, Hq, dtype=torch.bool, device=DEV)
    rest[1, 3] = False
    assert torch.equal(one[rest], ok[rest])


def test_append_captured_and_replayed():
    """Tokens stored one after another by a replayed graph (slots advance on the device), scales growing on the way:
    as eager calls do."""
    g = gen(15)
    Hq, Hkv, D, page, B = 4, 2, 128, 16, 3
    width = (Hq + 2 * Hkv) * D
    steps = (torch.randn(40, B, width, generator=g) * torch.exp2(torch.arange(40) % 7 - 3)[:, None, None]).to(torch.bfloat16).to(DEV)
    table = torch.from_numpy(S.rope_table(D, 64)).to(DEV)
    base = ints([0, 64, 128]).to(DEV)

    def fresh():
        c = S.KvCacheF8.empty(12, Hkv, page, D)
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            t.view(torch.uint8).fill_(0x30)
        return c

    a, b = fresh(), fresh()
    x, pos, slot = steps[0].clone(), ints([0] * B).to(DEV), base.clone()
    graph = torch.cuda.CUDAGraph()
    S.rope_append(x, Hq, fresh(), pos, slot, table)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q = S.rope_append(x, Hq, a, pos, slot, table)
        pos.add_(1)
        slot.add_(1)
    pos.zero_()
    slot.copy_(base)
    for t in range(40):
        x.copy_(steps[t])
        graph.replay()
        want = S.rope_append(steps[t], Hq, b, ints([t] * B).to(DEV), base + t, table)
        assert torch.equal(q, want), t
        for u, w in ((a.k, b.k), (a.v, b.v), (a.k_scale, b.k_scale), (a.v_scale, b.v_scale)):
            assert torch.equal(u.view(torch.uint8), w.view(torch.uint8)), t


@pytest.mark.parametrize("eps", [0.0, 1e-30])
def test_keys_of_heads_next_to_zero_and_huge(eps):
    """Norms of rows whose squares fp32 does not hold."""
    D = 64
    rows = torch.stack([torch.full((D,), 1e-38), torch.linspace(-1, 1, D) * 1e-30, torch.linspace(-1, 1, D) * 3e38,
                        torch.linspace(1, 2, D) * 1e-44])
    qkv = torch.cat([torch.ones(4, D), rows, rows], 1)
    w = torch.linspace(0.5, 2, D)
    k, s = torch.zeros(4, 1, 16, D), torch.full((4, 1, 1), 50, dtype=torch.uint8)
    cache = S.KvCacheF8(*[c.to(DEV) for c in (k.to(F.F8), k.to(F.F8), s, s.clone())])
    slots = [0, 16, 32, 48]
    S.rope_append(qkv.to(DEV), 1, cache, None, ints(slots).to(DEV), None, k_norm=w.to(DEV), eps=eps)
    y = rotate_all(rows[:, None], w, float(np.float32(eps)), None, None).float().double()
    codes, scale = F.store(k.double(), s, y, slots)
    assert torch.equal(cache.k_scale.cpu(), scale)
    F.same(cache.k, codes)


# ------------------------------------------------------------------ the linear in 8-bit integers

@pytest.mark.parametrize("M", [3, 70, 300])
def test_linear_weights_beyond_4_gb(M):
    K, N = 65536, 70000
    g = torch.Generator(DEV).manual_seed(2)
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8, device=DEV)
    x = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8, device=DEV)
    layer = S.I8Layer(K=K, N=N, s_hat_inv=None, Wq=w, sw=torch.ones(N, device=DEV))
    y, acc = S.linear_i8(x, torch.ones(M, device=DEV), layer, out_dtype=torch.float32, debug=True)
    some = [0, 1, 32767, 32768, 65535, 65536, N - 17, N - 2, N - 1]
    want = (x.double() @ w[some].double().t()).long()
    assert torch.equal(acc[:, some].long(), want) and torch.equal(y[:, some], want.float())


def test_linear_outputs_beyond_2_to_31():
    M, K, N = 33000, 64, 66000
    g = torch.Generator(DEV).manual_seed(2)
    x = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8, device=DEV)
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8, device=DEV)
    layer = S.I8Layer(K=K, N=N, s_hat_inv=None, Wq=w, sw=torch.ones(N, device=DEV))
    y = S.linear_i8(x, torch.ones(M, device=DEV), layer)
    rows, cols = [0, 16383, 32537, 32768, M - 1], [0, 255, 32768, 65535, N - 1]
    want = (x[rows].double() @ w[cols].double().t()).float().to(torch.bfloat16)
    assert torch.equal(y[rows][:, cols], want)
