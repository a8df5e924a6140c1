"""Plain 64-bit forms of the cache in 8 bits (E4M3 codes, a power of two for
each 16 tokens and head) for the tests. Nothing here comes from the library.

The definition fixes codes and scales bit for bit: a key y is taken in 64 bits
and rounded to fp32 once. Two 64-bit evaluations differ by about D 2^-53 of y,
so they round to different fp32 numbers once in 2^53 / (D 2^24) = 4 million
values and then to different codes once in 2^20 of those: codes are compared
for equality.
"""

from __future__ import annotations

import math

import torch

BLOCK, LEAST, MOST = 16, -117, 120
F8 = torch.float8_e4m3fn


def e4m3(x):
    """x (64 bits, |x| <= 448 or NaN) to the nearest E4M3 number, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.where(torch.isnan(x), x, torch.round(x / step) * step)


def exponent(m):
    """Least e >= LEAST with m <= 448 * 2^e (a float)."""
    if m == 0:
        return LEAST
    f, x = math.frexp(m / 448.0)           # (m / 448 is exact enough: fp32 numbers are 2^-24 apart, doubles 2^-53)
    return max(LEAST, x - 1 if f == 0.5 else x)


def values(codes, scale):
    """A cache's values in 64 bits: pages x heads x page x D."""
    x = codes.double().unflatten(2, (-1, BLOCK))
    return (x * torch.exp2(scale.double() - 127)[..., None, None]).flatten(2, 3)


def store(codes, scale, y, slot):
    """y (M x heads x D, 64 bits holding fp32 numbers) into copies of a cache (codes
    in 64 bits, scale), run of rows of one block by run: rows whose slot is
    outside store nothing. Returns (codes, scale)."""
    codes, scale = codes.clone(), scale.clone()
    pages, H, page, D = codes.shape
    M, t = y.shape[0], 0
    while t < M:
        s = int(slot[t])
        if not 0 <= s < pages * page:
            t += 1
            continue
        n = 1
        while t + n < M and int(slot[t + n]) // BLOCK == s // BLOCK:
            n += 1
        p, b = s // page, s % page // BLOCK
        i = [int(slot[r]) % BLOCK for r in range(t, t + n)]
        for h in range(H):
            new = y[t:t + n, h]
            finite = new[torch.isfinite(new)].abs()
            e = exponent(float(finite.max()) if finite.numel() else 0.0)
            block = codes[p, h, b * BLOCK:(b + 1) * BLOCK]
            if 0 not in i:
                old = min(max(int(scale[p, h, b]) - 127, LEAST), MOST)
                if old < e:
                    block[:] = e4m3(block * 2.0 ** max(old - e, -40))
                e = max(old, e)
            block[i] = e4m3(torch.where(torch.isfinite(new), new * 2.0 ** -e, float("nan")))
            scale[p, h, b] = e + 127
        t += n
    return codes, scale


def rotate(x, w, eps, table, pos, pair_axis, layout):
    """x: M x H x D, pos: axes x M: normed and rotated in 64 bits."""
    M, H, D = x.shape
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    y = x.clone()
    rot = 0 if table is None else table.shape[1]
    for t in range(M):
        for i in range(rot // 2):
            a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
            at = int(pos[pair_axis[i], t])
            c, s = float(table[at, i]), float(table[at, rot // 2 + i])
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return y


def same(got, want, what=""):
    """Codes (float8) against 64-bit numbers, NaN for NaN."""
    got = got.cpu().double()
    ok = (got == want) | (torch.isnan(got) & torch.isnan(want))
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.numel()} codes differ; first {got[~ok][:4]} for {want[~ok][:4]}"
