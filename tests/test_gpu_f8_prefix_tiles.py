"""serq_attn_decode_f8 on both sides of the rule that sends a shared prefix to
the LDS tiles: sequences x query heads x keys x D of 18 million x 128 or more, and
more than 64 rows to a key/value head."""

from __future__ import annotations

import pytest
import torch

from test_gpu_f8_cache import run_decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,prefix,Hq,Hkv,D,page", [
    (34, 22800, 48, 1, 64, 64),       # 1632 rows of heads of 64: tiles
    (33, 22700, 48, 1, 64, 64),       # a little less work: rows
    (17, 66200, 16, 4, 128, 16),      # 68 rows a head: tiles
    (16, 70400, 16, 4, 128, 16),      # 64: rows
])
def test_decode(B, prefix, Hq, Hkv, D, page):
    run_decode(B, [1 + 7 * (b % 4) for b in range(B - 1)] + [0], prefix, Hq, Hkv, D, page, torch.bfloat16)
