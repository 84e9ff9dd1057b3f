"""The choice rules (proj_plan.hpp, compiled for the host) over a sweep of sizes:
every kernel they take has a shape in the GPU tests that takes it too."""
import ctypes
import itertools
import os
import subprocess

import pytest

from choice_shapes import FFN16, FFN16_SLOW, FFN32, Q4_FEW, Q4_SLOW, Q4_TILES, ROPE

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
STRIPS_PATH, TILES_PATH = 3, 4  # of Q4Path
FFN_TILES = 5                   # of FfnPath
FLUSHES = (1, 2, 4)


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "plan_probe.so")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "segmented_gather_gemv_sgmv_amd", "csrc"), "-o", so,
                    os.path.join(HERE, "plan_probe.cpp")], check=True)
    return Rules(ctypes.CDLL(so))


class Rules:
    def __init__(self, dll):
        self.dll = dll

    def _tiles(self, M, N, batches, gated, flushes=0):
        out = (ctypes.c_int * 2)()
        self.dll.probe_tiles(ctypes.c_longlong(M), ctypes.c_longlong(N), batches, gated, flushes, out)
        return tuple(out)

    def q4(self, R, N, flushes, gated, nbytes=2, vec=1):
        """The kernels of a 4-bit call."""
        ll = ctypes.c_longlong
        path = self.dll.probe_q4_path(ll(R), ll(N), flushes, gated, nbytes, vec)
        detail = None
        if path == STRIPS_PATH:
            detail = self.dll.probe_q4_strip(ll(R), ll(N), flushes, gated)
        elif path == TILES_PATH:
            detail = self._tiles(R, N, 1, gated, flushes) if vec else "registers"
        return (nbytes, vec, gated, flushes, path, detail)

    def block(self, R, H, I, nbytes=2, vec=1, full=0):
        """The kernels of the gated block: forward, dx, the weights' gradients."""
        ll = ctypes.c_longlong
        path = self.dll.probe_ffn_path(ll(R), ll(I), nbytes, vec)
        ranges = ctypes.c_int()
        kind = self.dll.probe_sum(ll(R), ll(H), ll(I), 4 if full else 2, 0 if nbytes == 4 else 1,
                                  ctypes.byref(ranges))
        split = ranges.value > 1
        key = (nbytes, vec, full)
        if not vec:
            fwd = dx = dw = "registers"
        elif nbytes == 4:
            f32 = lambda M, N, b, g: self.dll.probe_f32_tiles(ll(M), ll(N), b, g)
            fwd, dx, dw = f32(R, I, 1, 1), kind, f32(I, H, 2, 0)
        else:
            fwd, dw = self._tiles(R, I, 1, 1), self._tiles(I, H, 2, 0)
            dx = kind if split else self._tiles(R, H, 1, 0)
        if path != FFN_TILES:
            fwd = self.dll.probe_ffn_wide(ll(I)) if path in (3, 4) else None
        return {key + ("forward", path, fwd), key + ("dx", split, dx), key + ("dW", dw)}

    def rope(self, R, heads, D, rot, interleaved, elem):
        V = 16 // elem
        vec = D % V == 0 and (rot if interleaved else rot // 2) % V == 0
        return (vec, interleaved,
                self.dll.probe_rope(ctypes.c_longlong(R), ctypes.c_longlong(heads), D, rot, interleaved,
                                    V if vec else 1))


ROWS = [1, 2, 3, 4, 5, 9, 16, 17, 24, 32, 33, 48, 64, 65, 80, 96, 97, 128, 150, 192, 225, 256, 257, 300, 400,
        520, 700, 1000, 1237, 1500, 2048, 2300, 3000, 4096, 5000, 8192]
SIZES = [8, 40, 100, 136, 200, 264, 520, 1000, 1504, 2048, 2800, 4096, 5504, 7500, 9500, 11008, 12500, 13824]


def test_every_q4_kernel_is_tested(rules):
    for gated, flushes in itertools.product((0, 1), FLUSHES):
        taken = {rules.q4(R, N, flushes, gated, *how) for R in ROWS for N in SIZES
                 for how in ((2, 1), (2, 0), (4, 1))}
        tested = {rules.q4(R, N, flushes, gated, nbytes) for R, N in Q4_FEW for nbytes in (2, 4)}
        tested |= {rules.q4(R, N, flushes, gated) for R, K, N in Q4_TILES}
        tested |= {rules.q4(R, N, flushes, gated, 2, 0) for R, K, N in Q4_SLOW}
        assert taken <= tested, sorted(taken - tested, key=str)
        # each kind of tile with several turns of the loop over K, too
        for kind in {k[5] for k in taken if k[4] == TILES_PATH and k[1]}:
            turns = [K for R, K, N in Q4_TILES if rules.q4(R, N, flushes, gated)[4:] == (TILES_PATH, kind)]
            assert max(turns) > 512, (gated, flushes, kind, turns)
    assert all(K % 8 == 0 for _, K, _ in Q4_TILES) and all(K % 8 for _, K, _ in Q4_SLOW)


def test_every_gated_kernel_is_tested(rules):
    taken, tested = set(), set()
    for R, H, I in itertools.product(ROWS, SIZES, SIZES):
        for how in ((2, 1), (2, 1, 1), (2, 0), (2, 0, 1), (4, 1)):
            taken |= rules.block(R, H, I, *how)
    for shapes, how in ((FFN16, (2, 1)), (FFN16, (2, 1, 1)), (FFN16_SLOW, (2, 0)), (FFN16_SLOW, (2, 0, 1)),
                        (FFN32, (4, 1))):
        for s in shapes:
            tested |= rules.block(*s, *how)
    assert taken <= tested, sorted(taken - tested, key=str)
    assert all(H % 8 == 0 and I % 8 == 0 for _, H, I in FFN16)
    assert all(H % 8 and I % 8 for _, H, I in FFN16_SLOW)


def test_every_rope_kernel_is_tested(rules):
    cases = lambda shapes: {rules.rope(R, h, D, rot, inter, elem) + (elem,) for R, h, D, rot in shapes
                            for inter in (0, 1) for elem in (2, 4)}
    sweep = [(R, h, D, rot) for R in (1, 8, 64, 500, 1024, 5000) for h in (1, 2, 8, 33, 40, 64, 96)
             for D in (2, 33, 64, 80, 128, 192, 256, 1024) for rot in (2, 30, 32, 64, 128) if rot <= D]
    taken, tested = cases(sweep), cases([(R, q + k, D, rot) for R, q, k, D, rot in ROPE])
    assert taken <= tested, sorted(taken - tested, key=str)
