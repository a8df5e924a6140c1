"""The attention block of examples/serve_attention.py with its cache in FP8
codes, its output projection in 8-bit integers and positions on three axes: the
calls together, as they are served."""

from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import f8_ref as F

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("serve_attention", os.path.join(ROOT, "examples", "serve_attention.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_graph_replays_equal_eager_steps_and_the_two_attentions_agree():
    ex = _example()
    outs, state = ex.serve(steps=20, codes=True)
    eager, state2 = ex.serve(steps=20, graph=False, codes=True)
    for a, b in zip(outs, eager):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)
    for a, b in zip(state["block"].tensors(), state2["block"].tensors()):
        used = state2["pages"].unique().long()
        written = a.view(torch.uint8)[used] == b.view(torch.uint8)[used]
        if a.dim() == 3:                                        # scales: those of blocks with tokens in them
            continue
        seen = torch.zeros(a.shape[0], a.shape[2], dtype=torch.bool, device="cuda")
        for row, n in zip(state2["pages"].tolist(), state2["kv_len"].tolist()):
            for t in range(n):
                seen[row[t // 16], t % 16] = True
        assert written.transpose(1, 2)[seen[used]].all()
    # Both calls round the weights and the result to bf16 over the same keys:
    # each is within 2^-8 (weights) + 2^-8 (result) of the exact value, relative
    # to the largest value in the cache that is attended to.
    block = state2["block"]
    v = F.values(block.cache.v.cpu(), block.cache.v_scale.cpu())[state2["pages"].long().cpu()]
    v = v.transpose(2, 3).flatten(1, 2)                          # users x tokens x heads x D
    seen = torch.arange(v.shape[1]) < state2["kv_len"].cpu()[:, None]
    top = float(v[seen].abs().max())
    assert ex.check(state2) <= 4 * 2.0 ** -8 * top
