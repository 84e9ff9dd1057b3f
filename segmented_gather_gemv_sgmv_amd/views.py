"""Which memory views [rows, heads, head_dim] with a dense last dimension take: outputs that
repeat their own elements, or that share some with another view, are refused with these.

Views of one fused buffer lie between each other without sharing an element, so ranges of
addresses alone cannot tell.  What strides tell is looked at first; where they leave it open,
every head's first address is compared.
"""
from __future__ import annotations

from . import _torch


def _reach(t, dims=(0, 1, 2)) -> int:
    """Elements from the first to behind the last along ``dims``."""
    return 1 + sum((t.shape[d] - 1) * t.stride(d) for d in dims)


def _starts(t):
    """Sorted distances in bytes of the heads' first elements from the view's."""
    torch = _torch()
    at = [torch.arange(t.shape[d]) * (t.stride(d) * t.element_size()) for d in (0, 1)]
    return (at[0][:, None] + at[1][None, :]).flatten().sort().values


def repeats(t) -> bool:
    """Whether two of the view's elements share memory."""
    reach = 1
    for step, n in sorted(zip(t.stride(), t.shape)):
        if n == 0:
            return False
        if n > 1:
            if step < reach:  # not nested: they may still lie between each other
                starts = _starts(t)
                return bool((starts[1:] - starts[:-1] < t.shape[2] * t.element_size()).any())
            reach += (n - 1) * step
    return False


def apart(a, b) -> bool:
    """Whether two views of one type share no element."""
    if a.numel() == 0 or b.numel() == 0:
        return True
    size = a.element_size()
    off = b.data_ptr() - a.data_ptr()
    if off >= _reach(a) * size or -off >= _reach(b) * size:
        return True
    # Equal steps along one dimension, within which both keep to places of their own.
    for d, other in ((0, (1, 2)), (1, (0, 2))):
        step = a.stride(d) * size
        if step and a.stride(d) == b.stride(d):
            at = off % step
            if _reach(a, other) * size <= at and at + _reach(b, other) * size <= step:
                return True
    torch = _torch()
    first, then = _starts(a), _starts(b) + off
    length = a.shape[2] * size, b.shape[2] * size
    before = torch.searchsorted(first, then + length[1]) - 1  # the last head of a that begins ahead of b's end
    return not bool(((before >= 0) & (first[before.clamp(min=0)] + length[0] > then)).any())
