"""Which memory views [rows, heads, head_dim] with a dense last dimension take: outputs that
repeat their own elements, or that share some with another view, are refused with these.

Views of one fused buffer lie between each other without sharing an element, so ranges of
addresses alone cannot tell.  What strides tell is looked at first; where they leave it open,
every head's first address is compared.  A view here is a tuple of plain numbers (address, rows,
heads, head_dim, row stride, head stride): a call has them in hand, and asking a tensor again for
each costs more than the arithmetic.
"""
from __future__ import annotations

from . import _torch


def view(t):
    """The view that a tensor is."""
    st = t.stride()
    return (t.data_ptr(), *t.shape, st[0], st[1])


def _starts(v):
    """Sorted distances in elements of the heads from the view's first."""
    torch = _torch()
    _, R, H, _, row, head = v
    count = lambda n: torch.arange(n, device="cpu")
    return (count(R)[:, None] * row + count(H)[None, :] * head).flatten().sort().values


def repeats(v) -> bool:
    """Whether two of the view's elements share memory."""
    _, R, H, D, row, head = v
    if R * H <= 1 or D == 0:
        return False
    if (H == 1 or head >= D) and (R == 1 or row >= (H - 1) * head + D):
        return False  # heads within rows
    if (R == 1 or row >= D) and (H == 1 or head >= (R - 1) * row + D):
        return False  # rows within heads
    starts = _starts(v)
    return bool((starts[1:] - starts[:-1] < D).any())


def apart(a, b, size: int) -> bool:
    """Whether two views of elements of ``size`` bytes share none."""
    pa, Ra, Ha, Da, ra, ha = a
    pb, Rb, Hb, Db, rb, hb = b
    if Ra * Ha * Da == 0 or Rb * Hb * Db == 0:
        return True
    off = pb - pa
    if off >= ((Ra - 1) * ra + (Ha - 1) * ha + Da) * size or -off >= ((Rb - 1) * rb + (Hb - 1) * hb + Db) * size:
        return True
    # Equal steps along one dimension, within which both keep to places of their own.
    if ra == rb and ra:
        at = off % (ra * size)
        if ((Ha - 1) * ha + Da) * size <= at and at + ((Hb - 1) * hb + Db) * size <= ra * size:
            return True
    if ha == hb and ha:
        at = off % (ha * size)
        if ((Ra - 1) * ra + Da) * size <= at and at + ((Rb - 1) * rb + Db) * size <= ha * size:
            return True
    first, then = _starts(a) * size, _starts(b) * size + off
    before = _torch().searchsorted(first, then + Db * size) - 1  # the last head of a that begins ahead of b's end
    return not bool(((before >= 0) & (first[before.clamp(min=0)] + Da * size > then)).any())
