"""What prefix_plan_bytes and prefix_attention_workspace_bytes reserve holds every way a batch may be cut (CPU),
and no partial results of rows that have none."""
import ctypes
import random

import pytest

from attention_plan_model import TARGET, cut, draw, reserved, widest
from test_attention_host import _cache, lib  # noqa: F401 (fixture)


@pytest.mark.parametrize("dim,dtype", [(64, 1), (96, 2), (128, 1), (128, 0), (256, 2)])
def test_room_for_every_cut(lib, dim, dtype):  # noqa: F811
    rng, most = random.Random(dim + dtype), 0.0
    for _ in range(1500):
        rows, tokens, cuts, prefix, rep, heads = draw(rng)
        if sum(rows) == 0:
            continue
        items, slots = cut(rows, tokens, cuts, prefix, rep, heads, widest(dim, dtype))
        T = sum(rows) + rng.choice([0, 0, 5])
        room = reserved(lib, _cache(heads=heads, dim=dim), T, len(rows), len(prefix), rep * heads, dtype)
        if room is None:
            continue
        assert items <= room[0] and slots <= room[1], (rows, tokens, cuts, prefix, rep, heads)
        most = max(most, slots / room[1])
    assert most > 0.5  # the bound is not far from what some of them take


def _bytes(lib, rows, seqs, prefixes, q_heads, heads, dim=128):  # noqa: F811
    cache = _cache(heads=heads, dim=dim)
    return lib.prefix_attention_workspace_bytes(ctypes.addressof(cache), rows, seqs, prefixes, q_heads, 2)


def test_no_room_for_what_is_not_joined(lib):  # noqa: F811
    """Without prefixes a batch's size does not count: only what is cut is joined."""
    for rows in (8192, 32768, 65536):
        assert _bytes(lib, rows, 5, 0, 32, 8) == _bytes(lib, 4096, 4, 0, 32, 8) <= (TARGET * 20 // 17 + 1) * 128 * 520
    assert _bytes(lib, 1, 1, 0, 32, 32) <= (TARGET * 20 // 17 + 1) * 16 * 520  # tiles of 16 rows
    # with one: a result from the prefix and one from the own tokens for every row and head, and little more
    for rows in (8192, 32768):
        assert _bytes(lib, rows, 5, 1, 32, 8) <= 2.1 * rows * 32 * 520 + 50e6
