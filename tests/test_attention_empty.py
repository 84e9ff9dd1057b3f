"""A plan of no rows or of no sequences has nothing to write (CPU)."""
import ctypes

from test_attention_host import FAKE, _cache, lib  # noqa: F401 (fixture)


def test_nothing_to_plan(lib):  # noqa: F811
    cache = _cache()
    p = ctypes.addressof(cache)
    for rows, seqs, prefixes in ((0, 4, 1), (6, 0, 0), (6, 0, 1), (0, 0, 0)):
        for plan in (None, FAKE):
            assert lib.prefix_plan(plan, 0, p, None, FAKE, 4, None, None, 4, rows, seqs, prefixes, 4, 1, None) == 0
        strides = (ctypes.c_int64 * 4)()
        assert lib.prefix_attention(None, None, None, p, None, None, 4, None, 4, rows, seqs, prefixes, 4, 1.0, strides, 1,
                                    None, 0, None) == 0
