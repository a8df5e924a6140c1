"""The attention half of a decoder layer as measured cases: rotating and storing
keys, prompt attention, single-token attention over a shared prefix.

Three operators stand between the quantized q/k/v linear and the quantized
output linear of a decoder layer when it serves:

append   takes the q/k/v linear's output, normalises each head's query and key
         (where the model does), rotates them by their position and writes the
         keys and values to their slots of a paged cache.
prefill  causal attention of packed new tokens of several sequences over that
         cache; query heads share key/value heads.
decode   one new token of every sequence of a batch over the cache; the batch
         may share a prefix, whose pages are named once.

``run`` computes them from elementary torch operations in 32 bits, or, with
``own`` set, through this repository's package. ``exact`` is their definition
in 64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
THETA = 500000.0


def listed():
    return [
        # a single user's next token: 48 head rows, all latency
        dict(name="append-1", op="append", M=1, Hq=32, Hkv=8, D=128, rot=128, layout="half", norm=False, page=16,
             dtype="bf16"),
        # a serving step of 61 sequences whose model rotates half of each head in neighbouring pairs, in 32 bits
        dict(name="append-61-part-f32", op="append", M=61, Hq=16, Hkv=16, D=64, rot=32, layout="interleaved",
             norm=True, page=32, dtype="f32"),
        # a long prompt's tokens with query and key norms
        dict(name="append-8192-norm", op="append", M=8192, Hq=32, Hkv=8, D=128, rot=128, layout="half", norm=True,
             page=16, dtype="bf16"),
        # a handful of short questions arriving together
        dict(name="prefill-short", op="prefill", B=7, lo=9, hi=157, old=0, Hq=32, Hkv=8, D=128, page=16, dtype="bf16"),
        # requests of mixed lengths packed into one step, 64 query heads
        dict(name="prefill-packed", op="prefill", B=8, lo=301, hi=4093, old=0, Hq=64, Hkv=8, D=128, page=16,
             dtype="bf16"),
        # one whole document
        dict(name="prefill-16384", op="prefill", B=1, lo=16384, hi=16384, old=0, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16"),
        # a chunk of new tokens in each of four conversations that already hold 12 thousand
        dict(name="prefill-chunk", op="prefill", B=4, lo=64, hi=256, old=12007, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16"),
        # a 32-bit model of 64-wide heads, a key/value head for each query head
        dict(name="prefill-f32", op="prefill", B=3, lo=500, hi=2000, old=0, Hq=16, Hkv=16, D=64, page=32, dtype="f32"),
        # a single user's next token over a middling context
        dict(name="decode-1", op="decode", B=1, lo=4095, hi=4095, prefix=0, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16"),
        # a batch of long conversations without anything in common
        dict(name="decode-ragged", op="decode", B=32, lo=513, hi=32000, prefix=0, Hq=64, Hkv=8, D=128, page=64,
             dtype="bf16"),
        # a busy service: one long instruction, 96 short dialogues after it
        dict(name="decode-prefix", op="decode", B=96, lo=5, hi=700, prefix=8209, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16"),
        # a 32-bit model of 64-wide heads with a short common instruction
        dict(name="decode-prefix-f32", op="decode", B=9, lo=33, hi=3000, prefix=777, Hq=16, Hkv=16, D=64, page=32,
             dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    Hq, Hkv = rng.choice([(32, 8), (32, 32), (64, 8), (16, 16), (8, 1), (24, 8), (16, 2)])
    c = dict(op=rng.choice(["append", "prefill", "decode"]), Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128, 128]),
             page=rng.choice([16, 16, 32, 64, 128]), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    if c["op"] == "append":
        c.update(M=_log(rng, 1, 8192), rot=rng.choice([c["D"], c["D"], c["D"] // 2, c["D"] // 4]),
                 layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.5)
        return c
    if c["op"] == "prefill":
        c.update(B=_log(rng, 1, 12), hi=_log(rng, 17, 6000), old=rng.choice([0, 0, _log(rng, 100, 9000)]))
        c["lo"] = max(1, int(c["hi"] * rng.uniform(0.05, 1.0)))
        # the plain form's padded scores stay below those of the largest listed case, those in 32 bits below a sixteenth
        most = (1 << 29) if c["dtype"] == "f32" else (1 << 32)
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


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    e, Hq, Hkv, D = _size(case), case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        M, row = case["M"], (Hq + 2 * Hkv) * D
        return {"bytes": M * (2 * row * e + 4 * case["rot"] + 8), "flops": M * (Hq + Hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    n = _lengths(case)
    if case["op"] == "prefill":
        old = case["old"]
        pairs = sum(k * old + k * (k + 1) // 2 for k in n)
        return {"bytes": e * D * sum(2 * k * Hq + 2 * (k + old) * Hkv for k in n), "flops": 4 * D * Hq * pairs}
    P = case["prefix"]
    return {"bytes": e * D * (2 * case["B"] * Hq + 2 * (sum(n) + P) * Hkv), "flops": 4 * D * Hq * sum(k + P for k in n)}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt, Hq, Hkv, D, page = _dtype(case), case["Hq"], case["Hkv"], case["D"], case["page"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dt)

    s = dict(case=case)
    if case["op"] == "append":
        M = case["M"]
        s["qkv"] = normal(M, (Hq + 2 * Hkv) * D)
        # one prompt's consecutive positions, or one position of each of M sequences
        start = int(torch.randint(0, 4096, (1,), generator=g, device=DEV))
        if M >= 256:
            s["pos"] = torch.arange(start, start + M, device=DEV, dtype=torch.int32)
        else:
            s["pos"] = torch.randint(0, 12288, (M,), generator=g, device=DEV, dtype=torch.int32)
        pages = (M + page - 1) // page + 5
        order = torch.randperm(pages, generator=g, device=DEV)
        if M >= 256:
            t = torch.arange(M, device=DEV)
            s["slot"] = (order[t // page] * page + t % page).to(torch.int32)
        else:
            s["slot"] = torch.randperm(pages * page, generator=g, device=DEV)[:M].to(torch.int32)
        f = THETA ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
        a = torch.arange(12288, device=DEV, dtype=torch.float64)[:, None] * f[None, :]
        s["table"] = torch.cat([a.cos(), a.sin()], 1).to(torch.float32)
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = 1 + 0.2 * torch.randn(D, generator=g, device=DEV)
            s["k_norm"] = 1 + 0.2 * torch.randn(D, generator=g, device=DEV)
        s["k"] = torch.zeros(pages, Hkv, page, D, device=DEV, dtype=dt)
        s["v"] = torch.zeros(pages, Hkv, page, D, device=DEV, dtype=dt)
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
    s["k"] = normal(pages, Hkv, page, D).mul_(gain.to(dt)).add_(bias.to(dt))
    s["v"] = normal(pages, Hkv, page, D)
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

def _rotate(x, cos, sin, layout):
    rot = 2 * cos.shape[-1]
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    c = s["case"]
    Hq, Hkv, D, page, dt = c["Hq"], c["Hkv"], c["D"], c["page"], _dtype(c)
    x = s["qkv"].view(c["M"], Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq].float(), x[:, Hq:Hq + Hkv].float(), x[:, Hq + Hkv:]
    if c["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * s["q_norm"]
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * s["k_norm"]
    t = s["table"][s["pos"].long()][:, None]
    cos, sin = t[..., :c["rot"] // 2], t[..., c["rot"] // 2:]
    at = s["slot"].long()
    s["k"][at // page, :, at % page] = _rotate(k, cos, sin, c["layout"]).to(dt)
    s["v"][at // page, :, at % page] = v
    return {"q": _rotate(q, cos, sin, c["layout"]).to(dt), "k": s["k"], "v": s["v"]}


def _dense(pages, table, length):
    """Pages of a cache in the order of `table` (... x n), as ... x heads x length x D in 32 bits."""
    x = pages[table.long()].float()                            # ... x n x heads x page x D
    x = x.transpose(-4, -3).flatten(-3, -2)                    # ... x heads x n page x D
    return x[..., :length, :].contiguous()


def _plain_prefill(s):
    c = s["case"]
    Hq, Hkv, D, B = c["Hq"], c["Hkv"], c["D"], c["B"]
    G, Lq, Lk, T = Hq // Hkv, s["max_q"], s["max_len"], s["q"].shape[0]
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(Lq, device=DEV)
    at = (cu[:-1, None] + i).clamp(max=T - 1)                  # B x Lq: the packed row of each padded one
    k, v = (_dense(s[x], s["page_table"], Lk) for x in ("k", "v"))
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
    k, v = (_dense(s[x], s["page_table"], L) for x in ("k", "v"))
    z = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(D ** -0.5)
    gone = torch.arange(L, device=DEV) >= s["kv_len"][:, None]
    z.masked_fill_(gone[:, None, None], float("-inf"))
    if P:
        pk, pv = (_dense(s[x], s["prefix"], P) for x in ("k", "v"))
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


def run(s):
    c = s["case"]
    if not own:
        return {"append": _plain_append, "prefill": _plain_prefill, "decode": _plain_decode}[c["op"]](s)
    import w4a4_linear_layers_amd as S
    cache = S.KvCache(s["k"], s["v"])
    if c["op"] == "append":
        q = S.rope_append(s["qkv"], c["Hq"], cache, s["pos"], s["slot"], s["table"], layout=c["layout"],
                          q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return {"q": q, "k": s["k"], "v": s["v"]}
    if c["op"] == "prefill":
        return S.attn_prefill(s["q"], s["cu_q"], cache, s["page_table"], s["kv_len"], max_len=s["max_len"])
    return S.attn_decode(s["q"], cache, s["page_table"], s["kv_len"], max_len=s["max_len"], prefix=s["prefix"],
                         prefix_len=c["prefix"])


# ------------------------------------------------------------------ the definition in 64 bits

def _attend(q, k, v, first):
    """q: rows x D over k, v: keys x D; row i sees the keys up to first + i (all of them where first is None)."""
    z = (q @ k.t()) / math.sqrt(q.shape[1])
    if first is not None:
        z = z.masked_fill(torch.ones_like(z, dtype=torch.bool).triu(first + 1), float("-inf"))
    return torch.softmax(z, 1) @ v


def exact(case, seed):
    s = prepare(case, seed)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    G = Hq // Hkv
    if case["op"] == "append":
        M, h = case["M"], case["rot"] // 2
        x = s["qkv"].double().view(M, Hq + 2 * Hkv, D)
        t = s["table"][s["pos"].long()].double()
        turn = torch.complex(t[:, :h], t[:, h:])[:, None]
        out = []
        for y, w in ((x[:, :Hq], s["q_norm"]), (x[:, Hq:Hq + Hkv], s["k_norm"])):
            if w is not None:
                y = y / (y.square().sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
            y = y.clone()
            pairs = y[..., :2 * h].unflatten(-1, (2, h)).transpose(-1, -2) if case["layout"] == "half" else y[..., :2 * h].unflatten(-1, (h, 2))
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            y[..., :2 * h] = (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)
            out.append(y)
        k, v = s["k"].double(), s["v"].double()
        flat = torch.stack([k, v]).transpose(2, 3).reshape(2, -1, Hkv, D)
        flat[0, s["slot"].long()], flat[1, s["slot"].long()] = out[1], x[:, Hq + Hkv:]
        k, v = flat.view(2, -1, page, Hkv, D).transpose(2, 3)
        return {"q": out[0], "k": k, "v": v}

    def keys(x, table, n, h):
        return x[table[:-(-n // page)].long(), h].reshape(-1, D)[:n].double()

    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    n = _lengths(case)
    if case["op"] == "prefill":
        at = 0
        for b, m in enumerate(n):
            for h in range(Hkv):
                k, v = (keys(s[x], s["page_table"][b], m + case["old"], h) for x in ("k", "v"))
                for j in range(h * G, h * G + G):
                    o[at:at + m, j] = _attend(s["q"][at:at + m, j].double(), k, v, case["old"])
            at += m
        return o
    for h in range(Hkv):
        lead = [keys(s[x], s["prefix"], case["prefix"], h) for x in ("k", "v")] if case["prefix"] else None
        for b, m in enumerate(n):
            k, v = (keys(s[x], s["page_table"][b], m, h) for x in ("k", "v"))
            if lead:
                k, v = torch.cat([lead[0], k]), torch.cat([lead[1], v])
            o[b, h * G:h * G + G] = _attend(s["q"][b, h * G:h * G + G].double(), k, v, None)
    return o
