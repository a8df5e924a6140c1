"""Plain 64-bit forms of the attention calls and how far fp32 kernels may be
from them, for the GPU tests. Nothing here comes from the library.

Tolerances. Let u = 2^-24 be the fp32 unit roundoff and U = 2^-8 (bf16) or 0
(fp32) that of the weights' type.

Attention: a score is a sum of D products, scaled: its error is at most
(D + 4) u scale sum_d |q_d k_d|; call e_z the largest such bound of a row. A
weight 2^z then has relative error at most e_z (1 + small) + 4 u, one u more
for every step that rescales the sums (at most one per 16 keys) and one for
every addition into them, and U for its rounding before the product with the
values. With A = sum p |v| / sum p the output is off by at most
    A (2 (e_z + (n / 8 + 64) u) + U) + U' |o|,
n the row's number of keys, U' the output type's roundoff (2^-8 or u).

Rotation: y = r w (x_a c - x_b s), r = 1 / sqrt(mean x^2 + eps) with relative
error at most (D / 2 + 6) u, and six roundings more: off by at most
    (D / 2 + 12) u r |w| (|x_a c| + |x_b s|) + U' |y|.
"""

from __future__ import annotations

import torch

U32 = 2.0 ** -24
UBF = 2.0 ** -8


def out_roundoff(dtype):
    return UBF if dtype == torch.bfloat16 else U32


def sequence(cache, pages, n, h):
    """The first n tokens of a row of page ids, head h: n x D in 64 bits."""
    ps = cache.shape[2]
    ids = pages[: -(-n // ps)].long()
    return cache[ids, h].reshape(-1, cache.shape[3])[:n].double()


def attend(q, k, v, scale):
    """One query row over all of k, v: (output, tolerance before the output's
    own rounding)."""
    n, D = k.shape
    if n == 0:
        return torch.zeros(D, dtype=torch.float64), torch.zeros(D, dtype=torch.float64)
    z = (k @ q) * scale
    p = torch.exp(z - z.max())
    p = p / p.sum()
    e_z = float((D + 4) * U32 * abs(scale) * (k.abs() @ q.abs()).max())
    A = p @ v.abs()
    return p @ v, A * 2 * (e_z + (n / 8 + 64) * U32), A


def attend_row(q, k, v, scale, dtype):
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], dtype=torch.float64)
        return z, z
    o, tol, A = attend(q, k, v, scale)
    if dtype == torch.bfloat16:
        tol = tol + A * UBF
    return o, tol + out_roundoff(dtype) * (o.abs() + tol) + 1e-30


def prefill(q, cu, k, v, table, kv_len, scale):
    """q: T x Hq x D (CPU), caches and tables on the CPU: (O, tolerance)."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    o = torch.zeros(T, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(o)
    for b in range(len(kv_len)):
        q0, q1, n = int(cu[b]), int(cu[b + 1]), int(kv_len[b])
        for h in range(Hq):
            ks, vs = sequence(k, table[b], n, h // G), sequence(v, table[b], n, h // G)
            for i in range(q0, q1):
                seen = max(0, n - (q1 - q0) + (i - q0) + 1)
                o[i, h], tol[i, h] = attend_row(q[i, h].double(), ks[:seen], vs[:seen], scale, q.dtype)
    return o, tol


def decode(q, k, v, table, kv_len, prefix, prefix_len, scale):
    B, Hq, D = q.shape
    G = Hq // k.shape[1]
    o = torch.zeros(B, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(o)
    for h in range(Hq):
        lead = [sequence(c, prefix, prefix_len, h // G) for c in (k, v)] if prefix_len else None
        for b in range(B):
            n = int(kv_len[b])
            ks, vs = sequence(k, table[b], n, h // G), sequence(v, table[b], n, h // G)
            if lead:
                ks, vs = torch.cat([lead[0], ks]), torch.cat([lead[1], vs])
            o[b, h], tol[b, h] = attend_row(q[b, h].double(), ks, vs, scale, q.dtype)
    return o, tol


def rotate(x, w, eps, table, pos, layout, dtype):
    """x: M x H x D of one kind (queries or keys): (y, tolerance) in 64 bits."""
    M, H, D = x.shape
    x = x.double()
    slack = 12.0
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
        slack += D / 2
    y, size = x.clone(), x.abs().clone()
    rot = 0 if table is None else table.shape[1]
    for t in range(M):
        for i in range(rot // 2):
            a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
            c, s = float(table[int(pos[t]), i]), float(table[int(pos[t]), rot // 2 + i])
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
            size[t, :, a] = (x[t, :, a] * c).abs() + (x[t, :, b] * s).abs()
            size[t, :, b] = (x[t, :, b] * c).abs() + (x[t, :, a] * s).abs()
    tol = slack * U32 * size
    return y, tol + out_roundoff(dtype) * (y.abs() + tol) + 1e-30


def check(got, want, tol, what=""):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    err = (got - want).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = int(torch.argmax(torch.where(torch.isnan(err), torch.full_like(err, 1e30), err - tol)))
        at = [int(x) for x in torch.unravel_index(torch.tensor(i), err.shape)]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; worst at {at}: got {got.flatten()[i]}, "
                             f"want {want.flatten()[i]} within {tol.flatten()[i]}")
