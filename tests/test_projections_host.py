"""Argument checks of the projections' entry points (CPU): every refusal
comes back before anything is enqueued."""
import os

import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg

FAKE = 0x1000  # non-null and aligned; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sg.LIBRARY):
        from segmented_gather_gemv_sgmv_amd import build
        build.build()
    return sg.lib()


def _weight(**kw):
    from segmented_gather_gemv_sgmv_amd.q4 import _CWeight
    return _CWeight(kw.get("tiles", FAKE), kw.get("meta", FAKE))


def _q4(lib, **kw):
    import ctypes
    w = kw.pop("w", _weight())
    a = dict(y=FAKE, x=FAKE, R=4, N=64, K=128, G=64, dt=1)
    a.update(kw)
    return lib.q4_linear(a["y"], a["x"], None if w is None else ctypes.addressof(w), None, a["R"],
                         a["N"], a["K"], a["G"], a["dt"], None)


def test_q4_linear_checks(lib):
    assert _q4(lib, dt=3) == 3
    for bad in (dict(N=0), dict(K=0), dict(G=0), dict(G=33), dict(G=-32), dict(R=-1)):
        assert _q4(lib, **bad) == 2, bad
    assert _q4(lib, K=(1 << 20) + 1) == 4
    assert _q4(lib, R=0, x=None, y=None, w=None) == 0
    for bad in (dict(y=None), dict(x=None), dict(w=None), dict(w=_weight(tiles=None)),
                dict(w=_weight(meta=None))):
        assert _q4(lib, **bad) == 1, bad
    assert _q4(lib, w=_weight(tiles=FAKE + 4)) == 4


def test_q4_gated_and_pack_checks(lib):
    import ctypes
    w = _weight()
    p = ctypes.addressof(w)
    call = lambda act=0, dt=2, g=p, h=FAKE: lib.q4_gated_ffn(h, FAKE, g, p, None, None, 4, 64, 128,
                                                           64, act, dt, None)
    assert call(act=5) == 2 and call(act=-1) == 2 and call(dt=7) == 3
    assert call(g=None) == 1 and call(h=None) == 1
    pack = lambda tiles=FAKE, meta=FAKE, G=64: lib.q4_pack(
        tiles, meta, FAKE, FAKE, None, 64, 128, G, 1, None)
    assert pack(tiles=None) == 1 and pack(meta=None) == 1 and pack(G=40) == 2
    assert lib.q4_tiles_bytes(17, 129) == 2 * 2 * 1024
    assert lib.q4_meta_bytes(17, 129, 64, 1) == 2 * 2 * 16 * 2 * 4
    assert lib.q4_meta_bytes(17, 129, 64, 0) == 2 * 2 * 16 * 2 * 8
    assert lib.q4_tiles_bytes(0, 5) == 0 and lib.q4_meta_bytes(4, 4, 31, 1) == 0


def test_gated_checks(lib):
    fwd = lambda h=FAKE, x=FAKE, R=4, H=64, I=64, act=0, dt=1: lib.gated_ffn(
        h, None, None, x, FAKE, FAKE, None, None, R, H, I, act, dt, None)
    assert fwd(dt=4) == 3 and fwd(H=0) == 2 and fwd(I=-1) == 2 and fwd(R=-2) == 2 and fwd(act=9) == 2
    assert fwd(h=None) == 1 and fwd(x=None) == 1 and fwd(R=0, h=None) == 0
    assert fwd(H=(1 << 20) + 1) == 4 and fwd(I=(1 << 20) + 1) == 4

    def bwd(dWg=FAKE, dWu=FAKE, dg=FAKE, x=FAKE, R=4, H=64, I=64, dt=1, ws=FAKE, ws_bytes=1 << 30):
        return lib.gated_ffn_backward(FAKE, dWg, dWu, dg, FAKE, FAKE, x, FAKE, FAKE, FAKE, FAKE, R,
                                      H, I, 0, dt, ws, ws_bytes, None)
    assert bwd(dt=-1) == 3 and bwd(R=-1) == 2
    assert bwd(dWg=None) == 1 and bwd(dWu=None) == 1 and bwd(dg=None) == 1 and bwd(x=None) == 1
    need = lib.gated_ffn_backward_workspace_bytes(300, 256, 4096, 1)
    assert need >= 2 * 300 * 256 * 4 and need % (300 * 256 * 4) == 0
    big = dict(R=300, H=256, I=4096)
    assert bwd(ws=None, **big) == 5 and bwd(ws_bytes=need - 1, **big) == 5 and bwd(ws=FAKE + 4, **big) == 5
    sizes = lib.gated_ffn_backward_workspace_bytes
    assert sizes(0, 256, 4096, 1) == 0 and sizes(300, 0, 4096, 1) == 0 and sizes(300, 256, 4096, 7) == 0
    assert sizes(8192, 8192, 4096, 1) == 0  # fills the chip by itself


def test_rope_checks(lib):
    import ctypes
    st = (ctypes.c_int64 * 8)(128, 64, 128, 64, 64, 64, 64, 64)

    def call(q=FAKE, pos=FAKE, pb=8, R=4, Hq=2, Hk=1, D=64, rot=64, strides=st, dt=1):
        return lib.rope(FAKE, FAKE, q, FAKE, pos, pb, FAKE, 1.0, R, Hq, Hk, D, rot, strides, 0, 0,
                        dt, None)
    assert call(dt=3) == 3
    for bad in (dict(R=-1), dict(Hq=-1), dict(D=0), dict(rot=0), dict(rot=63), dict(rot=66),
                dict(pb=2)):
        assert call(**bad) == 2, bad
    assert call(D=2048, rot=1026) == 4
    assert call(q=None) == 1 and call(pos=None) == 1 and call(strides=None) == 1
    assert call(R=0, q=None) == 0 and call(Hq=0, Hk=0) == 0


def test_python_refusals_without_a_gpu():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="must be on"):
        sg.gated_ffn(x, x, x)
    with pytest.raises(ValueError, match="must be on"):
        sg.q4_pack(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1))
    plan = sg.rope_plan(64, device="cpu")
    with pytest.raises(ValueError, match="on a GPU"):
        sg.rope(torch.zeros(2, 1, 64), None, torch.zeros(2, dtype=torch.int64), plan)
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=0.0),
                dict(rotary_dim=8, scaling=dict(kind="other", factor=2.0)),
                dict(rotary_dim=8, scaling=dict(kind="linear", factor=0.0)),
                dict(rotary_dim=8, scaling=dict(kind="by_parts", factor=2.0))):
        with pytest.raises(ValueError):
            sg.rope_plan(device="cpu", **bad)
    with pytest.raises(ValueError, match="layout"):
        sg.rope_plan(8, layout="thirds", device="cpu")


def test_by_parts_frequencies_end_to_end():
    f, m = sg.rope_frequencies(2)
    assert f == [1.0] and m == 1.0
