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
