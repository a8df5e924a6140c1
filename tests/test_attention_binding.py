"""The Python side of the attention calls on stand-in tensors (no GPU needed):
what it hands to the library, and what it refuses; and the library's bounds."""

from __future__ import annotations

import pytest
import torch

import w4a4_linear_layers_amd as S
from w4a4_linear_layers_amd import attention as A


class Fake:
    """As much of a device tensor as the calls look at."""

    made = 0

    def __init__(self, *shape, dtype=torch.bfloat16, device=0):
        Fake.made += 1
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device
        self.address = Fake.made << 20
        self.is_cuda, self.requires_grad = device >= 0, False
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def stride(self):
        return tuple(torch.Size(self.shape[i + 1:]).numel() for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.address

    def new_empty(self, shape):
        return Fake(*(shape if isinstance(shape, tuple) else (shape,)), dtype=self.dtype, device=self.index)


def ints(*shape, device=0):
    return Fake(*shape, dtype=torch.int32, device=device)


class Recorder:
    """Stands for the library: keeps the arguments of the last call and the
    device it was made on."""

    name, current = None, 0

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace"):
                return 64
            self.name, self.args, self.on = name, args, self.current
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(A, "lib", rec)
    monkeypatch.setattr(A, "_stream", lambda device: 70 + device)
    monkeypatch.setattr(A, "_current", lambda: rec.current, raising=False)

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, rec.current = rec.current, self.index

        def __exit__(self, *exc):
            rec.current = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    return rec


def cache(device=0):
    return S.KvCache(Fake(4, 2, 16, 64, device=device), Fake(4, 2, 16, 64, device=device))


def floats(*shape, device=0):
    return Fake(*shape, dtype=torch.float32, device=device)


def call_append(c, dtype=torch.bfloat16, d=0, **kw):
    a = dict(pos=ints(3, device=d), slot=ints(3, device=d), table=floats(9, 64, device=d),
             qkv=Fake(3, 8 * 64, dtype=dtype, device=d), cache=c, n_heads=4, q_norm=floats(64, device=d),
             k_norm=floats(64, device=d))
    return S.rope_append(**{**a, **kw})


def call_prefill(c, dtype=torch.bfloat16, d=0, **kw):
    a = dict(q=Fake(5, 4, 64, dtype=dtype, device=d), cu_q=ints(3, device=d), cache=c, page_table=ints(2, 3, device=d),
             kv_len=ints(2, device=d), max_len=40)
    return S.attn_prefill(**{**a, **kw})


def call_decode(c, dtype=torch.bfloat16, d=0, **kw):
    a = dict(q=Fake(2, 4, 64, dtype=dtype, device=d), cache=c, page_table=ints(2, 3, device=d),
             kv_len=ints(2, device=d), max_len=40, prefix=ints(1, device=d), prefix_len=16)
    return S.attn_decode(**{**a, **kw})


CALLS = [call_append, call_prefill, call_decode]


def handed(lib):
    """(k address, v address, pages, page size) of the last call."""
    a = lib.args
    return {"serq_rope_append": (a[-5], a[-4], a[-3], a[-2]), "serq_attn_prefill": a[9:13],
            "serq_attn_decode": a[7:11]}[lib.name]


@pytest.mark.parametrize("call", CALLS)
def test_a_replaced_cache_is_the_one_used(lib, call):
    c = cache()
    call(c)
    assert handed(lib) == (c.k.address, c.v.address, 4, 16)
    c.k, c.v = Fake(9, 2, 32, 64), Fake(9, 2, 32, 64)
    call(c)
    assert handed(lib) == (c.k.address, c.v.address, 9, 32)
    assert (c.n_pages, c.n_kv_heads, c.page_size, c.head_dim) == (9, 2, 32, 64)
    c.k.address += 4096                       # as set_ and resize_ may leave it
    call(c)
    assert handed(lib) == (c.k.address, c.v.address, 9, 32)


@pytest.mark.parametrize("call", CALLS)
def test_a_cache_replaced_in_part_is_refused(lib, call):
    c = cache()
    c.k = Fake(9, 2, 16, 64)
    with pytest.raises(ValueError):
        call(c)
    assert lib.name is None
    c.v = Fake(9, 2, 16, 64)
    call(c)
    c.k, c.v = (Fake(9, 2, 16, 64, dtype=torch.float32) for _ in range(2))
    with pytest.raises(ValueError):
        call(c)
    call(c, dtype=torch.float32)
    assert handed(lib)[:2] == (c.k.address, c.v.address)


ROWS = dict(qkv=Fake(3, 8 * 64, device=1), pos=ints(3, device=1), slot=ints(3, device=1), table=floats(9, 64, device=1),
            q_norm=floats(64, device=1), k_norm=floats(64, device=1), out=Fake(3, 4, 64, device=1))
PROMPT = dict(q=Fake(5, 4, 64, device=1), cu_q=ints(3, device=1), page_table=ints(2, 3, device=1),
              kv_len=ints(2, device=1), out=Fake(5, 4, 64, device=1), workspace=Fake(64, dtype=torch.uint8, device=1))
TOKEN = dict(q=Fake(2, 4, 64, device=1), page_table=ints(2, 3, device=1), kv_len=ints(2, device=1),
             prefix=ints(1, device=1), out=Fake(2, 4, 64, device=1), workspace=Fake(64, dtype=torch.uint8, device=1))
STRAY = [(c, k, v) for c, kw in zip(CALLS, (ROWS, PROMPT, TOKEN)) for k, v in kw.items()]


@pytest.mark.parametrize("call,name,tensor", STRAY, ids=[f"{c.__name__}-{k}" for c, k, _ in STRAY])
def test_a_tensor_on_another_device_is_refused(lib, call, name, tensor):
    with pytest.raises(ValueError):
        call(cache(), **{name: tensor})
    assert lib.name is None


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("current", [0, 1, 2])
def test_kernels_are_launched_on_the_cache_s_device(lib, call, current):
    lib.current = current
    call(cache(device=1), d=1)
    assert lib.on == 1 and lib.args[-1] == 71 and lib.current == current


def test_a_cache_on_two_devices_is_refused():
    with pytest.raises(ValueError):
        S.KvCache(Fake(4, 2, 16, 64), Fake(4, 2, 16, 64, device=1))


def wants_gradient(t):
    t.requires_grad = True
    return t


@pytest.mark.parametrize("call,name,tensor", [
    (call_append, "qkv", lambda: Fake(3, 8 * 64)), (call_append, "q_norm", lambda: floats(64)),
    (call_append, "k_norm", lambda: floats(64)), (call_prefill, "q", lambda: Fake(5, 4, 64)),
    (call_decode, "q", lambda: Fake(2, 4, 64))])
def test_a_gradient_is_not_lost_silently(lib, call, name, tensor):
    t = wants_gradient(tensor())
    with pytest.raises(ValueError, match="gradient"):
        call(cache(), **{name: t})
    assert lib.name is None
    with torch.no_grad():
        call(cache(), **{name: t})
    assert t.address in lib.args


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("which", ["k", "v"])
def test_a_cache_s_gradient_is_not_lost_silently(lib, call, which):
    c = cache()
    wants_gradient(getattr(c, which))
    with pytest.raises(ValueError, match="gradient"):
        call(c)
    with torch.inference_mode():
        call(c)
    assert lib.name is not None


@pytest.mark.parametrize("bf16,B,T,Hq,taken", [
    (1, 1, 1 << 30, 1, True), (1, 1 << 23, 1 << 23, 1, False), (1, (1 << 23) - (1 << 15) - 1, 1 << 23, 1, True),
    (1, 1 << 22, 1 << 22, 8, True), (0, 1, 1 << 29, 1, False), (0, 1, 1 << 28, 1, True),
    (0, 1 << 24, 1 << 24, 1, False), (0, 3, 1 << 24, 64, False)])
def test_prefills_of_more_than_one_launch_are_refused(bf16, B, T, Hq, taken):
    """On the host, before anything is launched (the addresses are never used)."""
    from w4a4_linear_layers_amd import _lib
    need = _lib.lib.serq_attn_prefill_workspace(bf16, B, T, Hq, 1, 64, 100)
    assert (need == 0) if taken else (need == -1)
    if not taken:
        a = 0x100000
        assert _lib.lib.serq_attn_prefill(a, bf16, 64 * Hq, a, B, T, Hq, 1, 64, a, a, 4, 16, a, 4, a, 100, 0.1, a,
                                          64 * Hq, None, 0, None) == _lib.SERQ_EINVAL


@pytest.mark.parametrize("call", [call_prefill, call_decode])
@pytest.mark.parametrize("max_len", [(1 << 30) + 1, 1 << 31, 1 << 32, (1 << 32) + 40, 1 << 63, -1, -(1 << 32) + 40])
def test_a_bound_that_no_int_holds_is_refused(lib, call, max_len):
    """(ctypes would hand on its low 32 bits)"""
    with pytest.raises(ValueError):
        call(cache(), max_len=max_len)
    assert lib.name is None
    assert S.attn_prefill_workspace(cache(), 2, 5, 4, max_len) == S.attn_decode_workspace(cache(), 2, 4, 0, max_len) == -1


def test_a_prefix_that_no_int_holds_is_refused(lib):
    for n in (-1, -(1 << 32) + 16, (1 << 32) + 16):
        with pytest.raises(ValueError):
            call_decode(cache(), prefix_len=n)
        assert S.attn_decode_workspace(cache(), 2, 4, n, 40) == -1
    assert lib.name is None
