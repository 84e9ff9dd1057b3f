"""Argument checks of the normed rotation, the cache and attention over it (CPU): every refusal
comes back before anything is enqueued."""
import ctypes
import os

import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from segmented_gather_gemv_sgmv_amd.kv import _CCache

FAKE = 0x1000  # non-null and aligned; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sg.LIBRARY):
        from segmented_gather_gemv_sgmv_amd import build
        build.build()
    return sg.lib()


def _cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=8, page=16, heads=2, dim=64, kind=0):
    return _CCache(k, v, ks, vs, pages, page, heads, dim, kind)


def test_norm_checks(lib):
    strides = (ctypes.c_int64 * 12)()
    call = lambda q=FAKE, qo=FAKE, k=FAKE, p=FAKE, f=FAKE, pb=8, eps=0.0, R=2, Hq=2, Hk=1, D=64, rot=64, st=strides, \
        dt=1: lib.qk_norm_rope(qo, FAKE, q, k, None, None, p, pb, f, 1.0, eps, R, Hq, Hk, D, rot, st, 0, dt, None)
    assert call(dt=3) == 3
    for bad in (dict(R=-1), dict(Hq=-1), dict(D=0), dict(rot=0), dict(rot=63), dict(rot=66), dict(pb=2), dict(eps=-1.0),
                dict(eps=float("nan"))):
        assert call(**bad) == 2, bad
    assert call(D=1025, rot=64) == 4 and call(Hq=65536) == 4
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(p=None), dict(f=None), dict(st=None)):
        assert call(**bad) == 1, bad
    assert call(R=0, q=None) == 0 and call(Hq=0, Hk=0, q=None) == 0
    need = lib.qk_norm_rope_backward_workspace_bytes(5000, 64, 64)
    assert need > 0 and lib.qk_norm_rope_backward_workspace_bytes(0, 64, 64) == 0
    back = lambda dw=FAKE, dy=FAKE, ws=FAKE, n=need, Hq=2, R=5000: lib.qk_norm_rope_backward(
        FAKE, FAKE, dw, None, dy, FAKE, FAKE, FAKE, None, None, FAKE, 8, FAKE, 1.0, 1e-6, R, Hq, 1, 64, 64, strides, 0, 1,
        ws, n, None)
    assert back(dy=None) == 1 and back(ws=None) == 5 and back(n=need - 1) == 5 and back(ws=FAKE + 4) == 5
    assert back(Hq=0, ws=None) == 5  # zero, but wanted: the sums run all the same


def test_cache_checks(lib):
    strides = (ctypes.c_int64 * 4)()

    def call(c, k=FAKE, v=FAKE, s=FAKE, sb=8, R=3, st=strides, dt=1, read=False):
        p = None if c is None else ctypes.addressof(c)
        if read:
            return lib.kv_read(k, v, p, s, sb, R, st, dt, None)
        return lib.kv_write(p, k, v, s, sb, R, st, dt, None)

    for read in (False, True):
        assert call(_cache(), dt=5, read=read) == 3 and call(None, read=read) == 1
        for bad in (dict(pages=0), dict(page=8), dict(page=24), dict(page=0), dict(heads=0), dict(dim=0), dict(kind=2)):
            assert call(_cache(**bad), read=read) == 2, bad
        for bad in (dict(dim=257), dict(heads=70000), dict(pages=2 ** 31 - 1, page=32)):
            assert call(_cache(**bad), read=read) == 4, bad
        for bad in (dict(k=None), dict(v=None), dict(ks=None), dict(vs=None)):
            assert call(_cache(**bad), read=read) == 1, bad
        assert call(_cache(k=FAKE + 8), read=read) == 4
        for bad in (dict(k=None), dict(v=None), dict(s=None), dict(st=None)):
            assert call(_cache(), read=read, **bad) == 1, bad
        assert call(_cache(), sb=2, read=read) == 2 and call(_cache(), R=-1, read=read) == 2
        assert call(_cache(), R=0, k=None, read=read) == 0
    # sizes: heads padded to 64, 96, 128, 192 or 256
    for dim, padded in ((1, 64), (64, 64), (65, 96), (97, 128), (129, 192), (193, 256), (256, 256)):
        assert lib.kv_codes_bytes(3, 32, 2, dim, 0) == 3 * 32 * 2 * padded
        assert lib.kv_codes_bytes(3, 32, 2, dim, 1) == 3 * 32 * 2 * padded // 2
        assert lib.kv_scales_bytes(3, 32, 2, dim, 0) == 3 * 32 * 2
        assert lib.kv_scales_bytes(3, 32, 2, dim, 1) == 3 * 32 * 2 * padded // 32
    assert lib.kv_codes_bytes(3, 20, 2, 64, 0) == 0 and lib.kv_codes_bytes(1, 16, 1, 300, 0) == 0


def test_attention_checks(lib):
    strides = (ctypes.c_int64 * 4)()
    c = _cache()
    p = ctypes.addressof(c)
    size = (6, 4, 1, 4, 1)
    nbytes, ws = lib.prefix_plan_bytes(p, *size), lib.prefix_attention_workspace_bytes(p, *size)
    assert nbytes > 0 and ws > 0
    for bad in ((-1, 4, 1, 4, 1), (6, -1, 1, 4, 1), (6, 4, -1, 4, 1), (6, 4, 1, 3, 1), (6, 4, 1, 0, 1), (6, 4, 1, 4, 9),
                (2 ** 31 - 1, 4, 1, 4, 1)):
        assert lib.prefix_plan_bytes(p, *bad) == 0 and lib.prefix_attention_workspace_bytes(p, *bad) == 0, bad

    def plan(plan=FAKE, n=nbytes, cache=p, lengths=FAKE, rows=FAKE, width=4, pl=FAKE, pi=None, pw=4, size=size):
        return lib.prefix_plan(plan, n, cache, lengths, rows, width, pl, pi, pw, *size, None)

    assert plan(cache=None) == 1 and plan(plan=None) == 1 and plan(lengths=None) == 1 and plan(pl=None) == 1
    assert plan(n=nbytes - 1) == 5 and plan(width=-1) == 2 and plan(pw=-1) == 2
    assert plan(rows=None, size=(3, 4, 1, 4, 1)) == 2  # fewer rows than sequences
    assert plan(size=(6, 4, 2, 4, 1)) == 2  # two prefixes, no runs
    assert plan(width=2 ** 27) == 4 and plan(pw=2 ** 27) == 4
    assert plan(size=(0, 4, 1, 4, 1), plan=None) == 0 or plan(size=(0, 4, 1, 4, 1)) == 0
    assert plan(size=(6, 0, 0, 4, 1), plan=None) == 0

    def attn(o=FAKE, q=FAKE, cache=p, plan=FAKE, pages=FAKE, width=4, pp=FAKE, pw=4, scale=1.0, st=strides, dt=1, w=FAKE,
             n=ws):
        return lib.prefix_attention(o, None, q, cache, plan, pages, width, pp, pw, 6, 4, 1, 4, scale, st, dt, w, n, None)

    for bad in (dict(o=None), dict(q=None), dict(cache=None), dict(plan=None), dict(pages=None), dict(pp=None), dict(st=None)):
        assert attn(**bad) == 1, bad
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(width=-1)):
        assert attn(**bad) == 2, bad
    for bad in (dict(w=None), dict(n=ws - 1), dict(w=FAKE + 8)):
        assert attn(**bad) == 5, bad
    assert attn(dt=4) == 3
    none = _cache(k=None)
    assert attn(cache=ctypes.addressof(none)) == 1


def test_python_refuses_the_cpu_and_dropped_gradients():
    cache = sg.kv_cache(2, 16, 1, 64, torch.float32, device="cpu")
    x, slots = torch.zeros(1, 1, 64), torch.zeros(1, dtype=torch.int64)
    plan = sg.rope_plan(64, device="cpu")
    i32 = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: sg.kv_write(cache, x, x, slots), lambda: sg.kv_read(cache, slots),
                 lambda: sg.qk_norm_rope(x, None, None, None, slots, plan),
                 lambda: sg.prefix_plan(cache, 1, i32[None], i32)):
        with pytest.raises(ValueError, match="must be on"):
            call()
    for kind, kw in ((ValueError, dict(kind="int8")), (ValueError, dict(page_size=17)), (ValueError, dict(num_pages=0)),
                     (ValueError, dict(head_dim=300)), (TypeError, dict(dtype=torch.float64))):
        args = dict(num_pages=2, page_size=16, kv_heads=1, head_dim=64, dtype=torch.float32, device="cpu")
        args.update(kw)
        with pytest.raises(kind):
            sg.kv_cache(**args)
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level():
        d = fwd.make_dual(x, torch.ones_like(x))
        with pytest.raises(RuntimeError, match="forward-mode"):
            sg.qk_norm_rope(d, None, None, None, slots, plan)
