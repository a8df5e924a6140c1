"""rope_append with positions on several axes on stand-in tensors (no GPU
needed): the name of the call that an error comes from, and the kinds of
sequences that name the axes."""

from __future__ import annotations

import array

import numpy as np
import pytest

import w4a4_linear_layers_amd as S
from test_attention_binding import cache, call_append, floats, ints, lib  # noqa: F401
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


@pytest.mark.parametrize("c", [cache, cache8])
@pytest.mark.parametrize("kind", [np.int64, np.int32, np.uint8, "array", "view", "strided", range])
def test_axes_in_any_sequence(lib, c, kind):  # noqa: F811
    """The numbers themselves are taken, whatever their width in memory."""
    axes = AXES
    if kind == "array":
        given = array.array("i", axes)
    elif kind == "view":
        given = memoryview(np.array(axes, np.int16))
    elif kind == "strided":
        given = np.array([[a, 3] for a in axes])[:, 0]
    elif kind is range:
        given, axes = range(1, 2), [1]
    else:
        given = np.array(axes, kind)
    n = max(axes) + 1
    table = {} if len(axes) == 32 else dict(table=floats(9, 2))
    call_append(c(), pair_axis=given, pos=ints(n, 3), **table)
    assert lib.args[14] == n and bytes(lib.args[15]) == bytes(axes)


@pytest.mark.parametrize("c", [cache, cache8])
@pytest.mark.parametrize("given", [32, np.int64(32), np.array([0, 1, 0, 1]), np.zeros(4, np.int64), array.array("i", [0] * 8), np.zeros((4, 8), np.uint8),
                                   [-1] * 32, [0.5] * 32, np.zeros(32), "a" * 32])
def test_what_names_no_axes_is_refused(lib, c, given):  # noqa: F811
    """A number is no sequence of so many zeros, and bytes of wider numbers are no axes."""
    with pytest.raises(ValueError):
        call_append(c(), pair_axis=given, pos=ints(1, 3))
    assert lib.name is None
