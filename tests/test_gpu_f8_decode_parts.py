"""serq_attn_decode_f8 over many sequences, whose keys are cut in larger parts:
each number of parts that the rule leaves, ragged lengths, heads and types."""

from __future__ import annotations

import pytest
import torch

from w4a4_linear_layers_amd import _lib
from test_gpu_f8_cache import run_decode

pytestmark = pytest.mark.gpu


def parts(dtype, B, Hq, Hkv, D, prefix, max_len):
    """Parts of a row, from the workspace: D sums, a maximum and a weight each."""
    size = _lib.lib.serq_attn_decode_f8_workspace(1 if dtype == torch.bfloat16 else 0, B, Hq, Hkv, D, prefix, max_len)
    return size // (4 * B * Hq * (D + 2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,Hq,Hkv,D,top,prefix,want", [
    (192, 4, 4, 64, 1500, 0, 3), (100, 16, 8, 128, 3000, 0, 6), (50, 32, 16, 64, 4096, 0, 6), (50, 16, 16, 128, 4000, 0, 6),
    (400, 4, 4, 64, 2000, 0, 3), (1600, 1, 1, 128, 2500, 0, 5), (2100, 2, 1, 64, 1100, 0, 3), (800, 1, 1, 64, 7000, 0, 7),
    (4100, 1, 1, 64, 1300, 0, 2), (200, 4, 4, 64, 900, 40, None)])
def test_decode(dtype, B, Hq, Hkv, D, top, prefix, want):
    lens = [max(0, int(top ** (b * 7919 % B / (B - 1))) - 1) for b in range(B - 1)] + [top]
    if want is not None:
        assert parts(dtype, B, Hq, Hkv, D, prefix, top) == want
    run_decode(B, lens, prefix, Hq, Hkv, D, 16, dtype)


def test_no_power_of_two_of_parts():
    for B in (96, 128, 200, 256, 300, 500, 999, 1024):
        for top in (1025, 1500, 2000, 2048, 3000, 4096, 5000, 8192, 16384, 100000, 1 << 20):
            n = parts(torch.bfloat16, B, 32, 8, 128, 0, top)
            assert n == 0 or n == 2 or n & (n - 1), (B, top, n)         # (0: one part, no workspace)
