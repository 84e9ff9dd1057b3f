"""Calls whose grids would pass 2^32 threads are refused before anything is enqueued (CPU)."""
import ctypes

from test_attention_host import FAKE, _cache, lib  # noqa: F401 (fixture)

UNSUPPORTED = 4


def test_attention(lib):  # noqa: F811
    for dim, lanes in ((64, 16), (128, 32), (256, 64)):
        cache = _cache(heads=1, dim=dim)
        p = ctypes.addressof(cache)
        rows = 2 ** 32 // lanes
        for sizes in (lib.prefix_plan_bytes, lib.prefix_attention_workspace_bytes):
            assert sizes(p, rows // 4, 1, 0, 4, 1) == 0 and sizes(p, rows // 4 - 100, 1, 0, 4, 1) > 0
        strides = (ctypes.c_int64 * 4)()
        assert lib.prefix_attention(FAKE, None, FAKE, p, FAKE, FAKE, 4, None, 0, rows // 4, 1, 0, 4, 1.0, strides, 1,
                                    FAKE, 2 ** 62, None) == UNSUPPORTED


def test_cache(lib):  # noqa: F811
    cache, strides = _cache(), (ctypes.c_int64 * 4)()
    p = ctypes.addressof(cache)
    for call in (lambda n: lib.kv_write(p, FAKE, FAKE, FAKE, 8, n, strides, 1, None),
                 lambda n: lib.kv_read(FAKE, FAKE, p, FAKE, 8, n, strides, 1, None)):
        assert call(2 ** 30) == UNSUPPORTED and call(2 ** 31 - 1) == UNSUPPORTED


def test_norm(lib):  # noqa: F811
    strides = (ctypes.c_int64 * 8)()
    call = lambda n: lib.qk_norm_rope(FAKE, FAKE, FAKE, FAKE, None, None, FAKE, 8, FAKE, 1.0, 1e-6, n, 2, 1, 64, 64,
                                      strides, 0, 1, None)
    assert call(2 ** 27) == UNSUPPORTED and call(2 ** 31 - 1) == UNSUPPORTED
