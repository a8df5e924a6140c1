"""Any tensor that requires a gradient is refused by the attention calls where
torch records gradients (stand-in tensors, no GPU needed)."""

from __future__ import annotations

import pytest
import torch

from test_attention_binding import Fake, cache, call_append, call_decode, call_prefill, floats, lib, wants_gradient  # noqa: F401
from test_f8_binding import cache8


@pytest.mark.parametrize("c", [cache, cache8])
@pytest.mark.parametrize("call,name,tensor", [
    (call_append, "table", lambda: floats(9, 64)), (call_append, "out", lambda: Fake(3, 4, 64)),
    (call_prefill, "out", lambda: Fake(5, 4, 64)), (call_decode, "out", lambda: Fake(2, 4, 64))])
def test_tables_and_outputs(lib, c, call, name, tensor):  # noqa: F811
    t = wants_gradient(tensor())
    with pytest.raises(ValueError, match="gradient"):
        call(c(), **{name: t})
    assert lib.name is None
    with torch.no_grad():
        call(c(), **{name: t})
    assert t.address in lib.args
