"""The example's cache in 8 bits after graph replays and after eager steps: the
scales of all blocks that hold tokens, and with them the values, are the same."""

from __future__ import annotations

import pytest
import torch

import f8_ref as F
from test_gpu_f8_example import _example

pytestmark = pytest.mark.gpu


def test_scales_and_values_after_replays_equal_those_of_eager_steps():
    ex = _example()
    _, state = ex.serve(steps=20, codes=True)
    _, eager = ex.serve(steps=20, graph=False, codes=True)
    assert torch.equal(state["pages"], eager["pages"]) and torch.equal(state["kv_len"], eager["kv_len"])
    a, b = state["block"].cache, eager["block"].cache
    page = a.page_size
    seen = torch.zeros(a.n_pages, page, dtype=torch.bool, device="cuda")
    for row, n in zip(eager["pages"].tolist(), eager["kv_len"].tolist()):
        for t in range(n):
            seen[row[t // page], t % page] = True
    begun = seen.view(a.n_pages, -1, F.BLOCK).any(-1)                # blocks with a token in them
    assert int(begun.sum()) >= 9
    for x, y, sx, sy in ((a.k, b.k, a.k_scale, b.k_scale), (a.v, b.v, a.v_scale, b.v_scale)):
        assert torch.equal(sx.transpose(1, 2)[begun], sy.transpose(1, 2)[begun])
        x, y = (F.values(c.cpu(), s.cpu()).transpose(1, 2)[seen.cpu()] for c, s in ((x, sx), (y, sy)))
        assert torch.equal(x, y) and torch.isfinite(x).all() and x.count_nonzero() > 0
