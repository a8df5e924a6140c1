"""The Python side of the attention calls on stand-in tensors (no GPU needed):
what it hands to the library, and what it refuses."""

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
        return Fake(*(shape if isinstance(shape, (tuple, torch.Size)) else (shape,)), dtype=self.dtype, device=self.index)


def ints(*shape, device=0):
    return Fake(*shape, dtype=torch.int32, device=device)


class Recorder:
    """Stands for the library: keeps the arguments of the last call."""

    name = None

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace"):
                return 64
            self.name, self.args = name, args
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(A, "lib", rec)
    monkeypatch.setattr(A, "_stream", lambda device: 7)
    return rec


def cache(pages=4, Hkv=2, page=16, D=64, dtype=torch.bfloat16, device=0):
    return S.KvCache(Fake(pages, Hkv, page, D, dtype=dtype, device=device), Fake(pages, Hkv, page, D, dtype=dtype, device=device))


def call_append(c, M=3, Hq=4, **kw):
    w = (Hq + 2 * 2) * 64
    dev = kw.pop("device", 0)
    dtype = kw.pop("dtype", torch.bfloat16)
    return S.rope_append(kw.pop("qkv", Fake(M, w, dtype=dtype, device=dev)), Hq, c, kw.pop("pos", ints(M)), kw.pop("slot", ints(M)),
                         kw.pop("table", Fake(9, 64, dtype=torch.float32)), **kw)


def call_prefill(c, T=5, B=2, **kw):
    return S.attn_prefill(kw.pop("q", Fake(T, 4, 64, dtype=kw.pop("dtype", torch.bfloat16))), kw.pop("cu_q", ints(B + 1)), c,
                          kw.pop("page_table", ints(B, 3)), kw.pop("kv_len", ints(B)), max_len=40, **kw)


def call_decode(c, B=2, **kw):
    return S.attn_decode(kw.pop("q", Fake(B, 4, 64, dtype=kw.pop("dtype", torch.bfloat16))), c, kw.pop("page_table", ints(B, 3)),
                         kw.pop("kv_len", ints(B)), max_len=40, **kw)


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
