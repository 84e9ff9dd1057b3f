"""A paged cache of K and V in 8 or 4 bits.

    cache = kv_cache(num_pages, 64, kv_heads, 128, torch.bfloat16, "fp8")  # zeroed, once
    kv_write(cache, k, v, slots)          # rows into token slots, quantized
    k, v = kv_read(cache, slots)          # and back

A slot is page * page_size + place in the page.  "fp8" keeps e4m3 codes with a power-of-two
scale per token and head, "fp4" e2m1 codes with one per 32 elements of a head
(include/sgmv.h has the rounding).  prefix_attention reads the cache as it lies.
No gradients: a cache serves.
"""
from __future__ import annotations

import ctypes

from . import _call_on, _check, _counts, _need, _no_gradients, _stream_ptr, _torch, dtype_code, lib
from .rotary import _heads, _position_types
from .views import apart, repeats, view

KINDS = {"fp8": 0, "fp4": 1}

_Strides4 = ctypes.c_int64 * 4


class _CCache(ctypes.Structure):
    """sgmv_kv_cache of sgmv.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("kind", ctypes.c_int32)]


class KVCache:
    """The device arrays of a cache and what they were made for (kv_cache)."""

    def __init__(self, arrays, num_pages, page_size, kv_heads, head_dim, dtype, kind):
        self.k, self.v, self.k_scales, self.v_scales = arrays
        self.num_pages, self.page_size = num_pages, page_size
        self.kv_heads, self.head_dim = kv_heads, head_dim
        self.dtype, self.kind, self.device = dtype, kind, self.k.device
        self._c = _CCache(*[t.data_ptr() for t in arrays], num_pages, page_size, kv_heads, head_dim,
                          KINDS[kind])
        self._ptr = ctypes.addressof(self._c)


def kv_cache(num_pages: int, page_size: int, kv_heads: int, head_dim: int, dtype, kind: str = "fp8",
             device="cuda") -> KVCache:
    """A zeroed cache of num_pages * page_size token slots for K and V [kv_heads,
    head_dim] in ``dtype``, kept as ``kind`` "fp8" or "fp4".  page_size is a multiple
    of 16, head_dim at most 256."""
    torch = _torch()
    if kind not in KINDS:
        raise ValueError(f"kind must be one of {', '.join(KINDS)}, got {kind!r}")
    dtype_code(dtype)
    sizes = (int(num_pages), int(page_size), int(kv_heads), int(head_dim))
    _counts(num_pages=sizes[0], page_size=sizes[1], kv_heads=sizes[2], head_dim=sizes[3])
    codes = lib().kv_codes_bytes(*sizes, KINDS[kind])
    scales = lib().kv_scales_bytes(*sizes, KINDS[kind])
    if not codes:
        raise ValueError("a cache needs at least one page and head, page_size a multiple of 16 and "
                         f"head_dim in 1..256, got {sizes}")
    arrays = [torch.zeros(n, dtype=torch.uint8, device=device) for n in (codes, codes, scales, scales)]
    return KVCache(arrays, *sizes, dtype, kind)


def _not_repeated(*outs):
    """Refuses an out [rows, heads, head_dim] whose elements share memory."""
    for o in outs:
        if repeats(view(o)):
            raise ValueError("out must not repeat its own elements")


def _rows(cache, t, name, n):
    st = _heads(t, name, cache.device, cache.dtype)
    if t.shape != (n, cache.kv_heads, cache.head_dim):
        raise ValueError(f"{name} must be {(n, cache.kv_heads, cache.head_dim)}, got {tuple(t.shape)}")
    return st[0], st[1]


def _slots(cache, slots):
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache (see kv_cache)")
    if slots.dtype not in _position_types():
        raise TypeError(f"slots must be int32 or int64, got {slots.dtype}")
    _need(slots, "slots", cache.device, None, 1)
    n = slots.shape[0]
    if n > 0x7FFFFFFF:
        _counts(rows=n)
    return n


def kv_write(cache: KVCache, k, v, slots) -> None:
    """Quantizes k and v [rows, kv_heads, head_dim] (any row and head strides) into the slots
    [rows] (int32 or int64).  A slot outside the cache, -1 for padding, skips its row.
    The slots of one call must differ: one named twice holds parts of either row."""
    n = _slots(cache, slots)
    _no_gradients("kv_write", k, v)
    strides = _Strides4(*_rows(cache, k, "k", n), *_rows(cache, v, "v", n))
    _check(_call_on(cache.device, lib().kv_write, cache._ptr, k.data_ptr(), v.data_ptr(), slots.data_ptr(),
                    slots.element_size(), n, strides, dtype_code(cache.dtype), _stream_ptr(cache.device)),
           "kv_write")


def kv_read(cache: KVCache, slots, out=None):
    """``(k, v)`` [rows, kv_heads, head_dim] of the slots [rows], in the cache's dtype; rows
    whose slot lies outside the cache are zeros.  ``out=(k, v)``, two tensors apart, receives them."""
    n, given = _slots(cache, slots), out is not None
    if not given:
        shape = (n, cache.kv_heads, cache.head_dim)
        out = tuple(_torch().empty(shape, dtype=cache.dtype, device=cache.device) for _ in range(2))
    else:
        _no_gradients("kv_read", *out)
    k, v = out
    strides = _Strides4(*_rows(cache, k, "out k", n), *_rows(cache, v, "out v", n))
    if given:
        _not_repeated(k, v)
        if not apart(view(k), view(v), k.element_size()):
            raise ValueError("out's k and v must lie apart")
    _check(_call_on(cache.device, lib().kv_read, k.data_ptr(), v.data_ptr(), cache._ptr, slots.data_ptr(),
                    slots.element_size(), n, strides, dtype_code(cache.dtype), _stream_ptr(cache.device)),
           "kv_read")
    return k, v
