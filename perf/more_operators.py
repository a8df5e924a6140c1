"""A decoder layer's 8-bit half as measured cases: rotary positions of several axes,
a cache of 8-bit codes with the attention that reads it, and the linear in
8-bit integers.

Five operators that a model calls when it serves:

turn     from the q/k/v linear's output to rotated queries and a filled cache, as for
         text, with a position on each of several axes (time, height, width) and
         each pair of a head turned by one of them.
append   the same into a cache of FP8 (E4M3) codes with a power of two for each 16
         tokens and head: a block whose largest value grows is recoded.
prefill  causal attention of packed new tokens over such a cache.
decode   one new token of every sequence of a batch over such a cache; the batch
         may share a prefix.
linear   int8 activations by int8 weights, a scale for each token and channel.

``run`` computes them from elementary torch operations, or, with ``own`` set,
through this repository's package. ``exact`` is their definition in 64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
THETA = 500000.0
BLOCK = 16                # tokens of a cache block
LEAST = -117              # least exponent of a block's scale
F8 = torch.float8_e4m3fn


def listed():
    return [
        # a token of a picture in a single conversation
        dict(name="turn-1", op="turn", M=1, Hq=32, Hkv=8, D=128, axes="16,24,24", cyclic=False, layout="half", norm=False,
             page=16, dtype="bf16"),
        # a clip's tokens: time, height and width taking turns among the pairs, heads normed
        dict(name="turn-5000-norm", op="turn", M=5000, Hq=32, Hkv=8, D=128, axes="24,20,20", cyclic=True, layout="half",
             norm=True, page=64, dtype="bf16"),
        # a serving step of 61 sequences, each somewhere in a block it has begun, in 32 bits
        dict(name="append-61-part-f32", op="append", M=61, Hq=16, Hkv=16, D=64, rot=32, layout="interleaved",
             norm=True, page=32, dtype="f32"),
        # a long prompt's tokens with query and key norms
        dict(name="append-8192-norm", op="append", M=8192, Hq=32, Hkv=8, D=128, rot=128, layout="half", norm=True,
             page=16, dtype="bf16"),
        # one whole document
        dict(name="prefill-12000", op="prefill", B=1, lo=12000, hi=12000, old=0, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16"),
        # a chunk of new tokens in each of four conversations that already hold 20 thousand
        dict(name="prefill-chunk", op="prefill", B=4, lo=64, hi=256, old=20011, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16"),
        # a single user's next token over a middling context
        dict(name="decode-1", op="decode", B=1, lo=7001, hi=7001, prefix=0, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16"),
        # a batch of long conversations without anything in common
        dict(name="decode-ragged", op="decode", B=48, lo=513, hi=40000, prefix=0, Hq=64, Hkv=8, D=128, page=64,
             dtype="bf16"),
        # a busy service: one long instruction, 120 short dialogues after it
        dict(name="decode-prefix", op="decode", B=120, lo=5, hi=900, prefix=6007, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16"),
        # one token through a gate/up layer kept in 8 bits
        dict(name="linear-1", op="linear", M=1, K=4096, N=28672, out="bf16"),
        # a decoding batch through a down layer
        dict(name="linear-45", op="linear", M=45, K=14336, N=4096, out="bf16"),
        # a prompt through a gate/up layer
        dict(name="linear-4000", op="linear", M=4000, K=4096, N=28672, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["turn", "append", "prefill", "decode", "linear"])
    if op == "linear":
        K, N = rng.choice([(4096, 4096), (4096, 6144), (4096, 28672), (14336, 4096), (8192, 10240), (8192, 8192), (1024, 992), (2048, 5000)])
        return dict(op=op, M=_log(rng, 1, 4000), K=K, N=N, out=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    Hq, Hkv = rng.choice([(32, 8), (32, 32), (64, 8), (16, 16), (8, 1), (24, 8), (16, 2)])
    c = dict(op=op, Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128, 128]), page=rng.choice([16, 16, 32, 64, 128]),
             dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    if op in ("turn", "append"):
        c.update(M=_log(rng, 1, 8192), layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.5)
        pairs = rng.choice([c["D"], c["D"], c["D"] // 2]) // 2
        if op == "append":
            c["rot"] = 2 * pairs
        else:
            a = pairs // 4 if rng.random() < 0.7 else rng.randint(1, pairs // 2)
            b = (pairs - a) // 2
            c.update(axes="%d,%d,%d" % (a, b, pairs - a - b), cyclic=rng.random() < 0.5)
        return c
    if op == "prefill":
        c.update(B=_log(rng, 1, 12), hi=_log(rng, 17, 6000), old=rng.choice([0, 0, _log(rng, 100, 9000)]))
        c["lo"] = max(1, int(c["hi"] * rng.uniform(0.05, 1.0)))
        # the plain form's padded scores stay below those of the largest listed case, those in 32 bits below a sixteenth
        most = (1 << 28) if c["dtype"] == "f32" else (1 << 32)
        while c["B"] * Hq * c["hi"] * (c["hi"] + c["old"]) > most:
            if c["B"] > 1:
                c["B"] -= 1
            else:
                c["hi"], c["old"] = max(1, c["hi"] * 3 // 4), c["old"] * 3 // 4
                c["lo"] = min(c["lo"], c["hi"])
        return c
    c.update(B=_log(rng, 1, 128), hi=_log(rng, 3, 20000), prefix=rng.choice([0, _log(rng, 40, 16000)]))
    c["lo"] = max(1, int(c["hi"] * rng.uniform(0.02, 1.0)))
    while c["B"] * Hkv * c["D"] * c["hi"] > 5e8:
        c["B"] -= 1
        if c["B"] <= 1:
            c["B"], c["hi"] = 1, c["hi"] // 2 + 1
            c["lo"] = min(c["lo"], c["hi"])
    return c


def _lengths(case):
    """The sequences' numbers of (new) tokens: evenly spread over the logarithm, in mixed order."""
    n, lo, hi = case["B"], case["lo"], case["hi"]
    v = [int(round(lo * (hi / lo) ** (i / (n - 1) if n > 1 else 1.0))) for i in range(n)]
    random.Random(n * 7919 + hi).shuffle(v)
    return v


def _pair_axis(case):
    """The axis that turns each pair: the axes' shares one after another, or taking turns until their shares are used."""
    left = [int(n) for n in case["axes"].split(",")]
    if not case["cyclic"]:
        return tuple(a for a, n in enumerate(left) for _ in range(n))
    got, a = [], 0
    while any(left):
        if left[a]:
            left[a] -= 1
            got.append(a)
        a = (a + 1) % len(left)
    return tuple(got)


def _rot(case):
    return case["rot"] if case["op"] == "append" else 2 * len(_pair_axis(case))


def _dtype(case):
    return torch.bfloat16 if case.get("dtype", case.get("out")) == "bf16" else torch.float32


def work(case):
    e = 2 if case.get("dtype", case.get("out")) == "bf16" else 4
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * e, "flops": 2 * M * N * K}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] in ("turn", "append"):
        M, rot, heads = case["M"], _rot(case), Hq + 2 * Hkv
        stored = e if case["op"] == "turn" else 1
        positions = 12 if case["op"] == "turn" else 4
        return {"bytes": M * (heads * D * e + Hq * D * e + 2 * Hkv * D * stored + 4 * rot + positions + 4),
                "flops": M * (Hq + Hkv) * (3 * rot + (4 * D if case["norm"] else 0))}
    n = _lengths(case)
    token = 2 * Hkv * (D + 1 / BLOCK)          # bytes of a token's keys and values
    if case["op"] == "prefill":
        old = case["old"]
        pairs = sum(k * old + k * (k + 1) // 2 for k in n)
        return {"bytes": sum(2 * k * Hq * D * e + (k + old) * token for k in n), "flops": 4 * D * Hq * pairs}
    P = case["prefix"]
    return {"bytes": 2 * case["B"] * Hq * D * e + (sum(n) + P) * token, "flops": 4 * D * Hq * sum(k + P for k in n)}


def _two_to(e, dtype=torch.float32):
    """2^e for whole e, exactly."""
    if dtype == torch.float32:
        return ((e.int() + 127) << 23).view(dtype)
    return ((e.long() + 1023) << 52).view(dtype)


def _coded(x):
    """Keys or values (pages x heads x page x D) as codes and block exponents."""
    y = x.float().unflatten(2, (-1, BLOCK))
    e = _exponent(y.abs().amax((-1, -2)))
    return (y * _two_to(-e)[..., None, None]).flatten(2, 3).to(F8), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = _dtype(case)
    s = dict(case=case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dt)

    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        # activations with a few strong channels, as int8 with each token's maximum at 127; weights likewise by channel
        x = torch.randn(M, K, generator=g, device=DEV)
        x[:, torch.randperm(K, generator=g, device=DEV)[:4]] *= 6.0
        m = x.abs().amax(1, keepdim=True)
        s["xq"] = torch.round(x * (127 / m)).to(torch.int8)
        s["sx"] = (m[:, 0] / 127).contiguous()
        w = torch.randn(N, K, generator=g, device=DEV)
        m = w.abs().amax(1, keepdim=True)
        s["wq"] = torch.round(w * (127 / m)).to(torch.int8)
        s["sw"] = (0.02 * m[:, 0] / 127).contiguous()
        return s
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    if case["op"] in ("turn", "append"):
        M, rot = case["M"], _rot(case)
        s["qkv"] = normal(M, (Hq + 2 * Hkv) * D)
        start = int(torch.randint(0, 4096, (1,), generator=g, device=DEV))
        t = torch.arange(M, device=DEV)
        many = M >= 256
        if case["op"] == "turn":
            # frames of 24 x 32 patches after some text, or patches of M sequences
            where = t if many else torch.randint(0, 8000, (M,), generator=g, device=DEV)
            s["pos"] = (start + torch.stack([where // 768, where % 768 // 32, where % 32])).to(torch.int32)
        elif many:
            s["pos"] = (start + t).to(torch.int32)
        else:
            s["pos"] = torch.randint(0, 12288, (M,), generator=g, device=DEV, dtype=torch.int32)
        # one prompt's consecutive tokens from the first of a page, or a token in a page of its own
        pages = ((M + page - 1) // page if many else M) + 5
        order = torch.randperm(pages, generator=g, device=DEV)
        if many:
            s["slot"] = (order[t // page] * page + t % page).to(torch.int32)
        else:
            s["slot"] = (order[:M] * page + torch.randint(0, page, (M,), generator=g, device=DEV)).to(torch.int32)
        f = THETA ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
        a = torch.arange(12288, device=DEV, dtype=torch.float64)[:, None] * f[None, :]
        s["table"] = torch.cat([a.cos(), a.sin()], 1).to(torch.float32)
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = 1 + 0.2 * torch.randn(D, generator=g, device=DEV)
            s["k_norm"] = 1 + 0.2 * torch.randn(D, generator=g, device=DEV)
        s["k"] = normal(pages, Hkv, page, D)
        s["v"] = normal(pages, Hkv, page, D)
        if case["op"] == "append":
            # (0.8: about half of the new tokens outgrow the block they come to)
            s["k"], s["k_scale"] = _coded(0.8 * s["k"])
            s["v"], s["v_scale"] = _coded(0.8 * s["v"])
        return s

    n = _lengths(case)
    prefill = case["op"] == "prefill"
    kv = [k + case["old"] for k in n] if prefill else n
    P = 0 if prefill else case["prefix"]
    need = [-(-k // page) for k in kv]
    wide, lead = max(max(need), 1), -(-P // page)
    pages = sum(need) + lead + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table, at = torch.zeros(len(n), wide, dtype=torch.int32, device=DEV), lead
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    s["prefix"] = order[:lead].contiguous() if P else None
    s["page_table"] = table
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    s["max_len"] = max(kv)
    # a few channels of the keys are much larger than the rest, with a mean, as after a trained projection
    bias = torch.randn(Hkv, 1, D, generator=g, device=DEV)
    gain = torch.ones(D, device=DEV)
    gain[torch.randperm(D, generator=g, device=DEV)[:4]] = 4.0
    s["k"], s["k_scale"] = _coded(normal(pages, Hkv, page, D).mul_(gain.to(dt)).add_(bias.to(dt)))
    s["v"], s["v_scale"] = _coded(normal(pages, Hkv, page, D))
    T = sum(n) if prefill else len(n)
    s["q"] = normal(T, Hq, D)
    if prefill:
        cu = [0]
        for k in n:
            cu.append(cu[-1] + k)
        s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["max_q"] = max(n)
    return s


# ------------------------------------------------------------------ plain forms

def _exponent(m):
    """The least e >= LEAST with m <= 448 * 2^e."""
    f, x = torch.frexp(m)
    return torch.where(m > 0, x - 9 + (f > 0.875), LEAST).clamp(min=LEAST)


def _turns(s):
    """Cosines and sines of each token: M x 1 x pairs."""
    if s["case"]["op"] == "turn":
        axis = torch.tensor(_pair_axis(s["case"]), device=DEV)
        half = axis.numel()
        pos, i = s["pos"].long()[axis].t(), torch.arange(half, device=DEV)      # M x pairs
        return s["table"][pos, i][:, None], s["table"][pos, half + i][:, None]
    t = s["table"][s["pos"].long()][:, None]
    return t.chunk(2, -1)


def _rotate(x, cos, sin, layout):
    rot = 2 * cos.shape[-1]
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _store(codes, scale, y, at, page):
    """y: M x heads x D in 32 bits to the slots `at` of a cache of codes."""
    M, H, D = y.shape
    per = page // BLOCK
    where, i = at // page, at % page // BLOCK
    block = where * per + i
    all_blocks = scale.transpose(1, 2).reshape(-1, H)                           # blocks x heads
    m = torch.zeros(all_blocks.shape, device=DEV)
    m.scatter_reduce_(0, block[:, None].expand(M, H), y.abs().amax(-1), "amax")
    begun = torch.zeros(all_blocks.shape[0], dtype=torch.int32, device=DEV)
    begun.scatter_reduce_(0, block, (at % BLOCK == 0).to(torch.int32), "amax")
    old, new = all_blocks[block].int() - 127, _exponent(m)[block]
    anew = begun[block, None] > 0
    e = torch.where(anew, new, torch.maximum(old, new))                         # M x heads
    d = torch.where(anew, 0, old - e)                                           # codes that are there: by 2^d
    if M < 256:       # each token's block
        x = codes.unflatten(2, (per, BLOCK))[where, :, i].float() * _two_to(d)[..., None, None]
        codes.unflatten(2, (per, BLOCK))[where, :, i] = x.to(F8)
    else:             # all blocks
        f = torch.ones(all_blocks.shape, device=DEV).index_copy_(0, block, _two_to(d))
        x = codes.unflatten(2, (per, BLOCK)).float() * f.view(-1, per, H).transpose(1, 2)[..., None, None]
        codes.copy_(x.flatten(2, 3).to(F8))
    codes[where, :, at % page] = (y * _two_to(-e)[..., None]).to(F8)
    scale[where, :, i] = (e + 127).to(torch.uint8)


def _plain_append(s):
    c = s["case"]
    Hq, Hkv, D, page, dt = c["Hq"], c["Hkv"], c["D"], c["page"], _dtype(c)
    x = s["qkv"].view(c["M"], Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq].float(), x[:, Hq:Hq + Hkv].float(), x[:, Hq + Hkv:]
    if c["op"] == "append":
        k = k.double()       # a key next to the border of two codes, or of two scales
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * s["q_norm"]
        k = k / torch.sqrt((k * k).mean(-1, keepdim=True) + EPS) * s["k_norm"]
    cos, sin = _turns(s)
    at = s["slot"].long()
    q, k = _rotate(q, cos, sin, c["layout"]).to(dt), _rotate(k, cos, sin, c["layout"])
    if c["op"] == "turn":
        s["k"][at // page, :, at % page] = k.to(dt)
        s["v"][at // page, :, at % page] = v
        return {"q": q, "k": s["k"], "v": s["v"]}
    _store(s["k"], s["k_scale"], k.float(), at, page)
    _store(s["v"], s["v_scale"], v.float(), at, page)
    return {"q": q, "k": s["k"], "k_scale": s["k_scale"], "v": s["v"], "v_scale": s["v_scale"]}


def _dense(codes, scale, table, length):
    """Pages of a cache in the order of `table` (... x n), as ... x heads x length x D in 32 bits."""
    x = codes[table.long()].float().unflatten(-2, (-1, BLOCK))                  # ... x n x heads x blocks x 16 x D
    x = x * _two_to(scale[table.long()].int() - 127)[..., None, None]
    x = x.flatten(-3, -2).transpose(-4, -3).flatten(-3, -2)                     # ... x heads x n page x D
    return x[..., :length, :].contiguous()


def _plain_prefill(s):
    c = s["case"]
    Hq, Hkv, D, B = c["Hq"], c["Hkv"], c["D"], c["B"]
    G, Lq, Lk, T = Hq // Hkv, s["max_q"], s["max_len"], s["q"].shape[0]
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(Lq, device=DEV)
    at = (cu[:-1, None] + i).clamp(max=T - 1)                  # B x Lq: the packed row of each padded one
    k, v = (_dense(s[x], s[x + "_scale"], s["page_table"], Lk) for x in ("k", "v"))
    q = s["q"].float()[at].view(B, Lq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Lq, D)
    z = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(D ** -0.5).view(B, Hkv, G, Lq, Lk)
    seen = torch.arange(Lk, device=DEV) <= (kv - n)[:, None, None] + i[:, None]
    seen &= (i < n[:, None])[:, :, None]
    z.masked_fill_(~seen[:, None, None], float("-inf"))
    z.sub_(z.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, Hkv, G * Lq, Lk), v).view(B, Hkv, G, Lq, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, Lq, Hq, D)
    return o[i < n[:, None]].to(_dtype(c))


def _plain_decode(s):
    c = s["case"]
    Hq, Hkv, D, B, P = c["Hq"], c["Hkv"], c["D"], c["B"], c["prefix"]
    G, L = Hq // Hkv, s["max_len"]
    q = s["q"].float().view(B, Hkv, G, D)
    k, v = (_dense(s[x], s[x + "_scale"], s["page_table"], L) for x in ("k", "v"))
    z = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(D ** -0.5)
    gone = torch.arange(L, device=DEV) >= s["kv_len"][:, None]
    z.masked_fill_(gone[:, None, None], float("-inf"))
    if P:
        pk, pv = (_dense(s[x], s[x + "_scale"], s["prefix"], P) for x in ("k", "v"))
        rows = q.transpose(0, 1).reshape(Hkv, B * G, D)
        y = torch.matmul(rows, pk.transpose(-1, -2).contiguous()).mul_(D ** -0.5)
        z = torch.cat([z, y.view(Hkv, B, G, P).transpose(0, 1)], -1)
    z = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-1e30))
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z[..., :L], v)
    if P:
        y = z[..., L:].transpose(0, 1).reshape(Hkv, B * G, P)
        o = o + torch.matmul(y, pv).view(Hkv, B, G, D).transpose(0, 1)
    return torch.where(total > 0, o / total, 0.0).view(B, Hq, D).to(_dtype(c))


def _plain_linear(s):
    acc = torch.matmul(s["xq"].float(), s["wq"].float().t())
    return (acc * s["sw"] * s["sx"][:, None]).to(_dtype(s["case"]))


def run(s):
    c = s["case"]
    if not own:
        return {"turn": _plain_append, "append": _plain_append, "prefill": _plain_prefill, "decode": _plain_decode,
                "linear": _plain_linear}[c["op"]](s)
    import w4a4_linear_layers_amd as S
    if c["op"] == "linear":
        layer = S.I8Layer(K=c["K"], N=c["N"], s_hat_inv=None, Wq=s["wq"], sw=s["sw"])
        return S.linear_i8(s["xq"], s["sx"], layer, out_dtype=_dtype(c))
    if c["op"] == "turn":
        q = S.rope_append(s["qkv"], c["Hq"], S.KvCache(s["k"], s["v"]), s["pos"], s["slot"], s["table"],
                          pair_axis=_pair_axis(c), layout=c["layout"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return {"q": q, "k": s["k"], "v": s["v"]}
    cache = S.KvCacheF8(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if c["op"] == "append":
        q = S.rope_append(s["qkv"], c["Hq"], cache, s["pos"], s["slot"], s["table"], layout=c["layout"],
                          q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return {"q": q, "k": s["k"], "k_scale": s["k_scale"], "v": s["v"], "v_scale": s["v_scale"]}
    if c["op"] == "prefill":
        return S.attn_prefill(s["q"], s["cu_q"], cache, s["page_table"], s["kv_len"], max_len=s["max_len"])
    return S.attn_decode(s["q"], cache, s["page_table"], s["kv_len"], max_len=s["max_len"], prefix=s["prefix"],
                         prefix_len=c["prefix"])


# ------------------------------------------------------------------ the definition in 64 bits

def _e4m3(x):
    """Nearest number of 4 significant bits (ties to even), from 2^-9 on a fixed grid; |x| <= 448."""
    step = _two_to(torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent - 4, torch.float64)
    return torch.round(x / step) * step


def _attend(q, k, v, first):
    """q: rows x D over k, v: keys x D; row i sees the keys up to first + i (all of them where first is None)."""
    z = (q @ k.t()) / math.sqrt(q.shape[1])
    if first is not None:
        z = z.masked_fill(torch.ones_like(z, dtype=torch.bool).triu(first + 1), float("-inf"))
    return torch.softmax(z, 1) @ v


def _exact_append(case, s):
    M, Hq, Hkv, D, page, rot = case["M"], case["Hq"], case["Hkv"], case["D"], case["page"], _rot(case)
    h = rot // 2
    x = s["qkv"].double().view(M, Hq + 2 * Hkv, D)
    axes = torch.tensor(_pair_axis(case) if case["op"] == "turn" else [0] * h, device=DEV)
    at = torch.atleast_2d(s["pos"].long()).t().gather(1, axes.expand(M, h))     # M x h
    turn = torch.complex(s["table"][:, :h].double().gather(0, at), s["table"][:, h:].double().gather(0, at))[:, None]
    out = []
    for y, w in ((x[:, :Hq], s["q_norm"]), (x[:, Hq:Hq + Hkv], s["k_norm"])):
        if w is not None:
            y = y / (y.square().sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
        y = y.clone()
        pairs = y[..., :rot].unflatten(-1, (2, h)).transpose(-1, -2) if case["layout"] == "half" else y[..., :rot].unflatten(-1, (h, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        y[..., :rot] = (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)
        out.append(y)
    got = {"q": out[0]}
    slot = s["slot"].long()
    for name, y in (("k", out[1]), ("v", x[:, Hq + Hkv:])):
        flat = s[name].double().transpose(1, 2).reshape(-1, Hkv, D)             # slots x heads x D
        if case["op"] == "append":
            y = y.float().double()
            e = s[name + "_scale"].transpose(1, 2).reshape(-1, Hkv).long() - 127
            blocks = flat.view(-1, BLOCK, Hkv, D) * _two_to(e, torch.float64)[:, None, :, None]   # values
            mine = slot // BLOCK
            top = torch.zeros(e.shape, dtype=torch.float64, device=DEV).scatter_reduce_(0, mine[:, None].expand(M, Hkv), y.abs().amax(-1), "amax")
            f, x2 = torch.frexp(top / 448)
            new = torch.where(top > 0, torch.where(f == 0.5, x2 - 1, x2), LEAST).clamp(min=LEAST).long()
            touched = torch.zeros(e.shape[0], device=DEV).index_fill_(0, mine, 1.0)[:, None] > 0
            fresh = torch.zeros(e.shape[0], device=DEV).index_fill_(0, mine[slot % BLOCK == 0], 1.0)[:, None] > 0
            e2 = torch.where(touched & fresh, new, torch.where(touched, torch.maximum(e, new), e))
            # what stands behind the values of a block begun anew stays as it is stored
            blocks = torch.where(fresh[:, None, :, None], blocks * _two_to(e2 - e, torch.float64)[:, None, :, None], blocks)
            flat = _e4m3(blocks / _two_to(e2, torch.float64)[:, None, :, None]).view(-1, Hkv, D)
            y = _e4m3(y / _two_to(e2, torch.float64)[mine][..., None])
            got[name + "_scale"] = None
        flat[slot] = y
        got[name] = flat.view(-1, page, Hkv, D).transpose(1, 2)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        # (sums of at most 14336 products of 8 bits are whole numbers below 2^53)
        return torch.matmul(s["xq"].double(), s["wq"].double().t()) * s["sx"].double()[:, None] * s["sw"].double()
    if case["op"] in ("turn", "append"):
        return _exact_append(case, s)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    G = Hq // Hkv

    def keys(x, table, n, h):
        ids = table[:-(-n // page)].long()
        y = s[x][ids, h].double().view(-1, BLOCK, D) * _two_to(s[x + "_scale"][ids, h].long() - 127, torch.float64).view(-1, 1, 1)
        return y.view(-1, D)[:n]

    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    n = _lengths(case)
    if case["op"] == "prefill":
        at = 0
        for b, m in enumerate(n):
            for h in range(Hkv):
                k, v = (keys(x, s["page_table"][b], m + case["old"], h) for x in ("k", "v"))
                for j in range(h * G, h * G + G):
                    o[at:at + m, j] = _attend(s["q"][at:at + m, j].double(), k, v, case["old"])
            at += m
        return o
    for h in range(Hkv):
        lead = [keys(x, s["prefix"], case["prefix"], h) for x in ("k", "v")] if case["prefix"] else None
        for b, m in enumerate(n):
            k, v = (keys(x, s["page_table"][b], m, h) for x in ("k", "v"))
            if lead:
                k, v = torch.cat([lead[0], k]), torch.cat([lead[1], v])
            o[b, h * G:h * G + G] = _attend(s["q"][b, h * G:h * G + G].double(), k, v, None)
    return o
