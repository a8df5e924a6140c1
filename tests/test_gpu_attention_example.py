"""The attention block of examples/serve_attention.py: the quantized linears
and the attention calls together, as they are served."""

from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("serve_attention", os.path.join(ROOT, "examples", "serve_attention.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_graph_replays_equal_eager_steps_and_the_two_attentions_agree():
    ex = _example()
    outs, state = ex.serve(steps=20)
    eager, state2 = ex.serve(steps=20, graph=False)
    for a, b in zip(outs, eager):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)
    # Both calls round the weights and the result to bf16 over the same keys:
    # each is within 2^-8 (weights) + 2^-8 (result) of the exact value, relative
    # to the largest value in the cache that is attended to.
    block = state2["block"]
    v = block.cache.v[state2["pages"].long()].transpose(2, 3).flatten(1, 2).float()      # users x tokens x heads x D
    seen = torch.arange(v.shape[1], device="cuda") < state2["kv_len"][:, None]
    top = float(v[seen].abs().max())
    assert ex.check(state2) <= 4 * 2.0 ** -8 * top
