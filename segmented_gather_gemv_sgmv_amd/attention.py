"""Attention of a batch over a quantized cache, a shared prefix read once for all.

    plan = prefix_plan(cache, q_heads, pages, lengths, prefix_pages=p, prefix_lengths=n)
    o = prefix_attention(q, cache, plan)          # every layer of the step

Sequence s holds lengths[s] tokens of its own in pages[s]; runs of sequences share a
prefix.  A row sees all of its run's prefix and its sequence's tokens up to itself
(include/sgmv.h has the details).  No gradients: this serves.
"""
from __future__ import annotations

import math

from . import _call_on, _check, _counts, _need, _no_gradients, _stream_ptr, _torch, dtype_code, lib
from .kv import KVCache, _not_repeated, _Strides4
from .rotary import _heads
from .views import apart, view


class PrefixPlan:
    """A step's work, cut up on the device (prefix_plan), with the tables it was made from."""

    def __init__(self, table, pages, prefix_pages, rows, seqs, prefixes, q_heads, cache, workspace_bytes,
                 ragged):
        self.table, self.pages, self.prefix_pages = table, pages, prefix_pages
        self.rows, self.seqs, self.prefixes, self.q_heads = rows, seqs, prefixes, q_heads
        self.ragged = ragged  # rows of no sequence are possible
        self.device, self.dtype, self.kind = cache.device, cache.dtype, cache.kind
        self.page_size, self.kv_heads, self.head_dim = cache.page_size, cache.kv_heads, cache.head_dim
        self.workspace_bytes = workspace_bytes


def _indices(t, name, dev, ndim):
    _need(t, name, dev, _torch().int32, ndim)
    return t


def prefix_plan(cache: KVCache, q_heads: int, pages, lengths, row_indptr=None, num_rows=None,
                prefix_pages=None, prefix_lengths=None, prefix_indptr=None) -> PrefixPlan:
    """Cuts a step's attention into work, on the device and without reading it back; serves every
    layer whose cache has ``cache``'s sizes, until lengths or rows change (page
    tables are read by prefix_attention itself).

    All tables are int32 on the cache's device: ``pages`` [sequences, width] and ``lengths``
    [sequences], tokens in the cache with this step's own; ``row_indptr`` [sequences + 1]
    with ``num_rows`` rows of q in all, or None for one row per sequence; ``prefix_pages`` [prefixes,
    width], ``prefix_lengths`` [prefixes] and ``prefix_indptr`` [prefixes + 1], the first sequence of
    every run and the end (None with one prefix: it is everyone's)."""
    torch = _torch()
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache (see kv_cache)")
    dev, q_heads = cache.device, int(q_heads)
    if q_heads < 1 or q_heads % cache.kv_heads:
        raise ValueError(f"q_heads must be a multiple of the cache's {cache.kv_heads} heads, got {q_heads}")
    S = _indices(lengths, "lengths", dev, 1).shape[0]
    if _indices(pages, "pages", dev, 2).shape[0] != S:
        raise ValueError(f"pages must be [{S}, width], got {tuple(pages.shape)}")
    if row_indptr is None:
        rows = S if num_rows is None else int(num_rows)
        if rows < S:
            raise ValueError(f"num_rows must be at least the {S} sequences, got {rows}")
    else:
        if _indices(row_indptr, "row_indptr", dev, 1).shape[0] != S + 1:
            raise ValueError(f"row_indptr must be [{S + 1}], got {tuple(row_indptr.shape)}")
        if num_rows is None:
            raise ValueError("row_indptr needs num_rows, the rows of q")
        rows = int(num_rows)
        if rows < 0:
            raise ValueError(f"num_rows must not be negative, got {rows}")
    G, prefix_width = 0, 0
    if prefix_pages is not None or prefix_lengths is not None:
        if prefix_pages is None or prefix_lengths is None:
            raise ValueError("prefix_pages and prefix_lengths go together")
        G = _indices(prefix_lengths, "prefix_lengths", dev, 1).shape[0]
        if _indices(prefix_pages, "prefix_pages", dev, 2).shape[0] != G:
            raise ValueError(f"prefix_pages must be [{G}, width], got {tuple(prefix_pages.shape)}")
        prefix_width = prefix_pages.shape[1]
    if prefix_indptr is not None:
        if _indices(prefix_indptr, "prefix_indptr", dev, 1).shape[0] != G + 1 or G == 0:
            raise ValueError(f"prefix_indptr must be [prefixes + 1] for {G} prefixes, got "
                             f"{tuple(prefix_indptr.shape)}")
    elif G > 1:
        raise ValueError("several prefixes need prefix_indptr")
    dt = dtype_code(cache.dtype)
    if max(rows, S, G, q_heads, pages.shape[1], prefix_width) > 0x7FFFFFFF:
        _counts(num_rows=rows, sequences=S, prefixes=G, q_heads=q_heads, pages_per_sequence=pages.shape[1],
                pages_per_prefix=prefix_width)
    sizes = (rows, S, G, q_heads, dt)
    nbytes = lib().prefix_plan_bytes(cache._ptr, *sizes)
    if not nbytes:
        raise ValueError(f"{rows} rows of {q_heads} heads over {S} sequences are more than a plan counts")
    table = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    ptr = lambda t: None if t is None else t.data_ptr()
    _check(_call_on(dev, lib().prefix_plan, table.data_ptr(), nbytes, cache._ptr, lengths.data_ptr(),
                    ptr(row_indptr), pages.shape[1], ptr(prefix_lengths), ptr(prefix_indptr), prefix_width,
                    *sizes, _stream_ptr(dev)), "prefix_plan")
    return PrefixPlan(table, pages, prefix_pages, rows, S, G, q_heads, cache,
                      lib().prefix_attention_workspace_bytes(cache._ptr, *sizes),
                      row_indptr is not None or rows > S)


def prefix_attention(q, cache: KVCache, plan: PrefixPlan, scale=None, out=None, lse=None):
    """o [rows, q_heads, D] = softmax(scale q K^T) V over every row's prefix and own tokens,
    ``scale`` 1 / sqrt(D) unless given.  q and ``out`` (optional, receives o, apart from q) may have any row
    and head strides; ``lse`` (optional, float32 [rows, q_heads]) receives the logarithms of the
    softmax's sums.  A row that sees no key is zeros, its lse minus infinity; rows of no sequence
    are not written (an ``out`` made here holds zeros for them).  A call allocates its workspace
    (``plan.workspace_bytes``): at most 36 MB without prefixes, with them about 1 KB more for every row
    and head of 128."""
    torch = _torch()
    if not isinstance(plan, PrefixPlan):
        raise TypeError("plan must be a PrefixPlan (see prefix_plan)")
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache (see kv_cache)")
    _no_gradients("prefix_attention", q, out, lse)
    dev, D = plan.device, plan.head_dim
    if (cache.device, cache.dtype, cache.kind, cache.page_size, cache.kv_heads, cache.head_dim) != (
            dev, plan.dtype, plan.kind, plan.page_size, plan.kv_heads, D):
        raise ValueError("the plan was made for a cache of other sizes")
    sq = _heads(q, "q", dev, cache.dtype)
    shape = (plan.rows, plan.q_heads, D)
    if q.shape != shape:
        raise ValueError(f"q must be {shape}, got {tuple(q.shape)}")
    scale = 1 / math.sqrt(D) if scale is None else float(scale)
    if not 0 < scale <= 2e38:
        raise ValueError(f"scale must be positive and at most 2e38, got {scale}")
    if out is None:
        out = (torch.zeros if plan.ragged else torch.empty)(shape, dtype=q.dtype, device=dev)
        so = (plan.q_heads * D, D)
    else:
        so = _heads(out, "out", dev, cache.dtype)
        if out.shape != shape:
            raise ValueError(f"out must be {shape}, got {tuple(out.shape)}")
        _not_repeated(out)
        if not apart(view(out), view(q), q.element_size()):
            raise ValueError("out must lie apart from q")
    if lse is not None:
        _need(lse, "lse", dev, torch.float32, 2)
        if lse.shape != shape[:2]:
            raise ValueError(f"lse must be {shape[:2]}, got {tuple(lse.shape)}")
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=dev)
    pages, prefix_pages = plan.pages, plan.prefix_pages
    _check(_call_on(
        dev, lib().prefix_attention, out.data_ptr(), None if lse is None else lse.data_ptr(), q.data_ptr(), cache._ptr,
        plan.table.data_ptr(), pages.data_ptr(), pages.shape[1],
        None if prefix_pages is None else prefix_pages.data_ptr(),
        0 if prefix_pages is None else prefix_pages.shape[1], plan.rows, plan.seqs, plan.prefixes,
        plan.q_heads, scale, _Strides4(sq[0], sq[1], so[0], so[1]), dtype_code(cache.dtype),
        ws.data_ptr(), plan.workspace_bytes, _stream_ptr(dev)), "prefix_attention")
    return out
