"""The attention calls read a cache's scales by words of 4 bytes: a cache made by
the package ends with a whole one, whatever its number of blocks."""

from __future__ import annotations

import pytest
import torch

import w4a4_linear_layers_amd as S
from w4a4_linear_layers_amd import attention as A


@pytest.mark.parametrize("pages,heads,page", [(1, 1, 16), (5, 1, 16), (2, 1, 16), (3, 3, 64), (4, 2, 32), (7, 1, 32), (1, 1, 1024)])
def test_scales_end_with_a_whole_word(monkeypatch, pages, heads, page):
    """(on the host: only the tensors' making is looked at)"""
    monkeypatch.setattr(A.KvCacheF8, "_now", lambda self: None)
    c = S.KvCacheF8.empty(pages, heads, page, 64, device="cpu")
    for s in (c.k_scale, c.v_scale):
        assert s.shape == (pages, heads, page // 16) and s.dtype == torch.uint8 and s.is_contiguous()
        assert s.untyped_storage().nbytes() % 4 == 0 and s.storage_offset() == 0
        assert 0 <= s.untyped_storage().nbytes() - s.numel() < 4
