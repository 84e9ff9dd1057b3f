"""The scale's range (CPU): scores are taken times scale log2(e), which has to be a finite float32."""
import ctypes

from test_attention_host import FAKE, _cache, lib  # noqa: F401 (fixture)


def test_scales(lib):  # noqa: F811
    cache, strides = _cache(), (ctypes.c_int64 * 4)()
    p = ctypes.addressof(cache)
    call = lambda scale, rows=6: lib.prefix_attention(FAKE, None, FAKE, p, FAKE, FAKE, 4, FAKE, 4, rows, 4, 1, 4, scale,
                                                      strides, 1, FAKE, 2 ** 40, None)
    for scale in (2.4e38, 2.9e38, 3.4e38, 1e39, 1e-46):  # the last two leave float32
        assert call(scale) == 2, scale
    assert call(2e38, rows=0) == 0 and call(1e-38, rows=0) == 0
