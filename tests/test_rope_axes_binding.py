"""rope_append with positions on several axes on stand-in tensors (no GPU
needed): the name of the call that an error comes from, and the kinds of
sequences that name the axes."""

from __future__ import annotations

import pytest

import w4a4_linear_layers_amd as S
from test_attention_binding import cache, call_append, ints, lib  # noqa: F401
from test_f8_binding import cache8

AXES = [0] * 8 + [1] * 12 + [2] * 12


@pytest.mark.parametrize("c,kw,name", [
    (cache, dict(), "serq_rope_append"), (cache, dict(pair_axis=AXES), "serq_rope_append_axes"),
    (cache, dict(pair_axis=bytes(32)), "serq_rope_append_axes"), (cache8, dict(), "serq_rope_append_f8"),
    (cache8, dict(pair_axis=AXES), "serq_rope_append_f8")])
def test_an_error_names_the_call_that_was_made(lib, monkeypatch, c, kw, name):  # noqa: F811
    called = []
    for n in ("serq_rope_append", "serq_rope_append_axes", "serq_rope_append_f8"):
        monkeypatch.setattr(lib, n, lambda *a, n=n: called.append(n) or -1, raising=False)
    if kw:
        kw = dict(kw, pos=ints(3 if kw["pair_axis"] is AXES else 1, 3))
    with pytest.raises(S.SerqError) as e:
        call_append(c(), **kw)
    assert called == [name] and str(e.value).startswith(name + " failed")
