"""The attention half of a decoder layer (include/serq.h): argument
marshalling only. Every online call enqueues the library's HIP kernels on the
current torch stream.

    cache = KvCache.empty(n_pages, n_kv_heads, page_size, head_dim)
    table = torch.from_numpy(rope_table(head_dim, max_pos, theta=5e5)).cuda()
    q = rope_append(qkv, n_heads, cache, pos, slot, table)           # queries; keys and values stored
    o = attn_prefill(q, cu_q, cache, pages, kv_len, max_len=...)     # new tokens, packed
    o = attn_decode(q, cache, pages, kv_len, max_len=...)            # one token per sequence

For inference: none of these calls has a backward pass. Where torch records
gradients, a tensor that requires one is refused rather than its gradient
lost; under torch.no_grad() it is taken.
"""

from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from . import _lib
from ._lib import SERQ_BF16, SERQ_EINVAL, SERQ_F32, SerqError, check

lib = _lib.lib
try:
    import torch
except ImportError:  # pragma: no cover - library use without PyTorch
    torch = None

_BF16, _F32, _I32 = (getattr(torch, name, None) for name in ("bfloat16", "float32", "int32"))
_MOST_KEYS = 1 << 30     # (a larger int would reach the library by its low 32 bits)
_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "bands": 3}


def _no_gradient(what):
    if torch.is_grad_enabled():
        raise ValueError(f"{what} requires a gradient, and the attention calls have none: use torch.no_grad()")


@dataclass
class KvCache:
    """Paged keys and values: two contiguous device tensors, each (pages, kv
    heads, page size, head dim), of one dtype. Slot s is token s % page size
    of page s // page size. They may be replaced, by larger ones say: every
    call takes the tensors as they are then (a captured graph keeps those of
    its capture)."""

    k: "object"
    v: "object"

    def __post_init__(self):
        self._now()

    def _now(self):
        """What a call needs of the tensors, checked and read afresh: (k
        address, v address, pages, kv heads, page size, head dim, torch dtype,
        library dtype, device index). Kept from an earlier call, an address
        could be of memory that is another tensor's by now."""
        k, v = self.k, self.v
        shape, dtype, dev = k.shape, k.dtype, k.get_device()
        if len(shape) != 4 or v.shape != shape or v.dtype is not dtype or v.get_device() != dev:
            raise ValueError("k and v must be (pages, kv heads, page size, head dim) tensors alike")
        if dev < 0 or not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("device tensors must be contiguous CUDA tensors")
        if dtype is _BF16:
            code = SERQ_BF16
        elif dtype is _F32:
            code = SERQ_F32
        else:
            raise ValueError("the cache must be float32 or bfloat16")
        if k.requires_grad or v.requires_grad:
            _no_gradient("the cache")
        pages, heads, page, D = shape
        return k.data_ptr(), v.data_ptr(), pages, heads, page, D, dtype, code, dev

    n_pages = property(lambda self: self._now()[2])
    n_kv_heads = property(lambda self: self._now()[3])
    page_size = property(lambda self: self._now()[4])
    head_dim = property(lambda self: self._now()[5])
    torch_dtype = property(lambda self: self._now()[6])
    dtype = property(lambda self: self._now()[7])
    pointers = property(lambda self: self._now()[:2])

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, *, dtype=None, device="cuda"):
        """A cache of uninitialised pages (bfloat16 unless ``dtype`` says otherwise)."""
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        dtype = torch.bfloat16 if dtype is None else dtype
        return cls(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device))


def rope_table(rot_dim: int, max_pos: int, *, theta: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
               orig_len: int = 0, low: float = 1.0, high: float = 4.0, mscale: float = 1.0) -> np.ndarray:
    """Cosines and sines of the rotary embedding (serq_rope_table), host:
    (max_pos, rot_dim) float32, each row its cosines, then its sines.
    ``scaling`` is "plain", "linear", "base" or "bands"."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    if rot_dim < 0 or max_pos < 0:
        raise SerqError("serq_rope_table", SERQ_EINVAL, "sizes must be positive")
    t = np.empty((max_pos, rot_dim), np.float32)
    check("serq_rope_table", lib.serq_rope_table(rot_dim, max_pos, theta, _SCALINGS[scaling], factor, orig_len, low,
                                                 high, mscale, t.ctypes.data if t.size else None))
    return t


# The handle of a device's current stream. torch.cuda.current_stream() builds
# a Stream object around it, which takes longer than the smallest of these
# kernels.
_stream = getattr(getattr(torch, "_C", None), "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
# The device that kernels are launched on. A call makes the cache's device the
# current one where it is not: a stream's handle alone does not say it (the
# default stream's is 0 on every device).
_current = getattr(getattr(torch, "_C", None), "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())


# The checks below run on every call of a decoding step, where a handful of
# microseconds is what the kernels take: each attribute is read once.

def _ints(t, shape, dev, what):
    if t.dtype is not _I32 or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA int32 tensor of shape {tuple(shape)} on the cache's device")
    return t.data_ptr()


def _rows(t, shape, D, dtype, dev, what):
    """Row stride of a (rows, heads, head dim) tensor whose rows are whole."""
    if len(shape) != 3:
        raise ValueError(f"{what} must be (rows, heads, head dim)")
    n, h, d = shape
    if d != D or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{what} must be a CUDA (rows, heads, {D}) tensor of the cache's dtype and device")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != d and h > 1):
        raise ValueError(f"{what}: heads must lie one after another in a row")
    return s0 if n > 1 else h * d


def _out(out, shape, dtype, dev):
    """(output, its row stride)"""
    if out.shape != shape:
        raise ValueError(f"out must be of shape {tuple(shape)}")
    return out, _rows(out, shape, shape[2], dtype, dev, "out")


def _space(workspace, need, q, dev):
    """(tensor that holds it, address, bytes) of a workspace that is needed"""
    if need < 0:
        raise ValueError("sizes that the library does not take")
    if workspace is None:
        workspace = q.new_empty((need + 3) // 2)       # (of q's type: at least two bytes each)
        return workspace, workspace.data_ptr(), need
    size = workspace.numel() * workspace.element_size()
    if workspace.get_device() != dev or not workspace.is_contiguous() or size < need:
        raise ValueError(f"workspace must be a contiguous CUDA tensor of {need} bytes or more on the cache's device")
    return workspace, workspace.data_ptr(), size


def _norm(w, D, dev):
    if w.dtype is not _F32 or w.shape != (D,) or w.get_device() != dev or not w.is_contiguous():
        raise ValueError(f"norms must be contiguous CUDA float32 tensors of {D} on the cache's device")
    if w.requires_grad:
        _no_gradient("a norm")
    return w.data_ptr()


def rope_append(qkv, n_heads: int, cache: KvCache, pos, slot, table, *, layout: str = "half", q_norm=None, k_norm=None,
                eps: float = 1e-6, out=None):
    """Queries of the q/k/v linear's output, with keys and values stored in
    the cache (serq_rope_append), on the current stream. ``qkv`` is M x
    (n_heads + 2 kv heads) * head dim (unit column stride), ``pos`` and
    ``slot`` M int32, ``table`` (max_pos, rot_dim) float32 on the device or
    None for no rotation. Returns M x n_heads x head dim."""
    kc, vc, n_pages, Hkv, page, D, tdt, dt, dev = cache._now()
    if dev != _current():
        with torch.cuda.device(dev):
            return rope_append(qkv, n_heads, cache, pos, slot, table, layout=layout, q_norm=q_norm, k_norm=k_norm,
                               eps=eps, out=out)
    shape = qkv.shape
    if len(shape) != 2 or qkv.get_device() != dev or qkv.dtype is not tdt:
        raise ValueError("qkv must be a two-dimensional CUDA tensor of the cache's dtype and device")
    if qkv.requires_grad:
        _no_gradient("qkv")
    M, width = shape
    ld, unit = qkv.stride()
    if width != (n_heads + 2 * Hkv) * D or (unit != 1 and M > 0):
        raise ValueError(f"qkv must have {(n_heads + 2 * Hkv) * D} columns of unit stride")
    if M <= 1:
        ld = width
    order = _LAYOUTS.get(layout)
    if order is None:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}")
    rot = max_pos = 0
    tp = pp = None
    if table is not None:
        size = table.shape
        if len(size) != 2 or table.dtype is not _F32 or table.get_device() != dev or not table.is_contiguous():
            raise ValueError("table must be a contiguous CUDA (max_pos, rot_dim) float32 tensor on the cache's device")
        max_pos, rot = size
        if rot:
            tp, pp = table.data_ptr(), _ints(pos, (M,), dev, "pos")
    qw = None if q_norm is None else _norm(q_norm, D, dev)
    kw = None if k_norm is None else _norm(k_norm, D, dev)
    sp = _ints(slot, (M,), dev, "slot")
    q, ldq = (qkv.new_empty((M, n_heads, D)), n_heads * D) if out is None else _out(out, (M, n_heads, D), tdt, dev)
    status = lib.serq_rope_append(
        qkv.data_ptr(), dt, ld, M, n_heads, Hkv, D, qw, kw, eps, tp, rot, max_pos, order, pp,
        sp, q.data_ptr(), ldq, kc, vc, n_pages, page, _stream(dev))
    if status:
        check("serq_rope_append", status)
    return q


def attn_prefill_workspace(cache: KvCache, B: int, T: int, n_heads: int, max_len: int) -> int:
    """Bytes of workspace attn_prefill needs (serq_attn_prefill_workspace);
    -1 for sizes that it does not take."""
    _, _, _, Hkv, _, D, _, dt, _ = cache._now()
    if not 0 <= max_len <= _MOST_KEYS:
        return -1
    return lib.serq_attn_prefill_workspace(dt, B, T, n_heads, Hkv, D, max_len)


def attn_prefill(q, cu_q, cache: KvCache, page_table, kv_len, *, max_len: int, scale: float | None = None, out=None,
                 workspace=None):
    """Causal attention of packed new tokens over the cache
    (serq_attn_prefill) on the current stream. ``q`` is T x heads x head dim,
    ``cu_q`` B + 1, ``page_table`` B x pages and ``kv_len`` B int32 on the
    device; ``max_len`` bounds kv_len; ``scale`` is head_dim ** -0.5 unless
    given. A workspace is taken from torch's allocator unless given. Returns
    T x heads x head dim."""
    kc, vc, n_pages, Hkv, page, D, tdt, dt, dev = cache._now()
    if dev != _current():
        with torch.cuda.device(dev):
            return attn_prefill(q, cu_q, cache, page_table, kv_len, max_len=max_len, scale=scale, out=out,
                                workspace=workspace)
    if q.requires_grad:
        _no_gradient("q")
    shape = q.shape
    ldq = _rows(q, shape, D, tdt, dev, "q")
    T, Hq, _ = shape
    if not 0 <= max_len <= _MOST_KEYS:
        raise ValueError("max_len must be 0 to 2^30")
    if page_table.dim() != 2:
        raise ValueError("page_table must be sequences x pages")
    pages = page_table.shape
    B = pages[0]
    tp = _ints(page_table, pages, dev, "page_table")
    cp = _ints(cu_q, (B + 1,), dev, "cu_q")
    kp = _ints(kv_len, (B,), dev, "kv_len")
    o, ldo = (q.new_empty(shape), Hq * D) if out is None else _out(out, shape, tdt, dev)
    size = lib.serq_attn_prefill_workspace(dt, B, T, Hq, Hkv, D, max_len)
    hold = wp = None
    if size:
        hold, wp, size = _space(workspace, size, q, dev)
    status = lib.serq_attn_prefill(
        q.data_ptr(), dt, ldq, cp, B, T, Hq, Hkv, D, kc, vc, n_pages, page, tp, pages[1], kp,
        max_len, D ** -0.5 if scale is None else scale, o.data_ptr(), ldo, wp, size, _stream(dev))
    if status:
        check("serq_attn_prefill", status)
    return o


def attn_decode_workspace(cache: KvCache, B: int, n_heads: int, prefix_len: int, max_len: int) -> int:
    """Bytes of workspace attn_decode needs (serq_attn_decode_workspace); -1
    for sizes that it does not take."""
    _, _, _, Hkv, _, D, _, dt, _ = cache._now()
    if not 0 <= max_len <= _MOST_KEYS or not 0 <= prefix_len <= _MOST_KEYS:
        return -1
    return lib.serq_attn_decode_workspace(dt, B, n_heads, Hkv, D, prefix_len, max_len)


def attn_decode(q, cache: KvCache, page_table, kv_len, *, max_len: int, prefix=None, prefix_len: int = 0,
                scale: float | None = None, out=None, workspace=None):
    """One new token per sequence over the cache (serq_attn_decode) on the
    current stream. ``q`` is B x heads x head dim; ``page_table`` B x pages
    and ``kv_len`` B int32 give each sequence's own tokens, ``prefix`` (int32
    page ids) and ``prefix_len`` the tokens that all of them share before
    those. Returns B x heads x head dim."""
    kc, vc, n_pages, Hkv, page, D, tdt, dt, dev = cache._now()
    if dev != _current():
        with torch.cuda.device(dev):
            return attn_decode(q, cache, page_table, kv_len, max_len=max_len, prefix=prefix, prefix_len=prefix_len,
                               scale=scale, out=out, workspace=workspace)
    if q.requires_grad:
        _no_gradient("q")
    shape = q.shape
    ldq = _rows(q, shape, D, tdt, dev, "q")
    B, Hq, _ = shape
    if not 0 <= max_len <= _MOST_KEYS or not 0 <= prefix_len <= _MOST_KEYS:
        raise ValueError("max_len and prefix_len must be 0 to 2^30")
    pages = page_table.shape
    if len(pages) != 2 or pages[0] != B:
        raise ValueError(f"page_table must be {B} x pages")
    tp = _ints(page_table, pages, dev, "page_table")
    kp = _ints(kv_len, (B,), dev, "kv_len")
    pp = None
    if prefix_len > 0:
        need = -(-prefix_len // page)
        if prefix is None or prefix.numel() < need:
            raise ValueError(f"prefix must hold {need} page ids")
        pp = _ints(prefix, (prefix.numel(),), dev, "prefix")
    o, ldo = (q.new_empty(shape), Hq * D) if out is None else _out(out, shape, tdt, dev)
    size = lib.serq_attn_decode_workspace(dt, B, Hq, Hkv, D, prefix_len, max_len)
    hold = wp = None
    if size:
        hold, wp, size = _space(workspace, size, q, dev)
    status = lib.serq_attn_decode(
        q.data_ptr(), dt, ldq, B, Hq, Hkv, D, kc, vc, n_pages, page, pp, prefix_len, tp,
        pages[1], kp, max_len, D ** -0.5 if scale is None else scale, o.data_ptr(), ldo, wp, size, _stream(dev))
    if status:
        check("serq_attn_decode", status)
    return o
