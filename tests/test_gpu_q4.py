"""q4_linear and q4_gated_ffn against their plain 64-bit forms."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from proj_helpers import (DTYPES, F32, check, gated_forward, half_step, make_q4, q4_parts,
                          q4_product, tiny)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TILE_ROWS = 256  # 16-bit calls of more rows round the scaled weights (include/sgmv.h)

# rows, in, out, group: single tokens, ragged and odd sizes, groups longer than
# the row, tiles with and without a K remainder, sizes no vector fits.
SHAPES = [
    (1, 32, 16, 32), (1, 4096, 64, 128), (5, 1000, 333, 32), (16, 256, 48, 64), (17, 384, 100, 128),
    (33, 131, 51, 32), (64, 513, 72, 64), (3, 96, 40, 96), (2, 200, 24, 512), (1, 1, 1, 32),
    (130, 640, 80, 160), (256, 264, 40, 64),
]
TILE_SHAPES = [(257, 640, 264, 128), (300, 200, 136, 64), (400, 333, 77, 32), (513, 1152, 129, 96),
               (300, 64, 300, 32), (1100, 264, 4000, 128), (1100, 328, 4000, 64), (700, 136, 6000, 32),
               (2100, 130, 100, 64), (900, 392, 1000, 32)]


def _x(gen, R, K, dtype):
    return torch.randn(R, K, generator=gen).to(dtype).to(DEV)


def _linear(R, K, N, G, dt, zeros, bias, seed=0):
    gen = torch.Generator().manual_seed(seed)
    dtype = DTYPES[dt]
    w = make_q4(gen, N, K, G, dtype, zeros, DEV)
    x = _x(gen, R, K, dtype)
    b = torch.randn(N, generator=gen).to(dtype).to(DEV) if bias else None
    y = sg.q4_linear(x, sg.q4_pack(*w, group_size=G, in_features=K), bias=b)
    ref, bound = q4_product(x, w, K, G, R > TILE_ROWS and dt != "f32")
    if bias:
        ref = ref + b.double().cpu()
        bound = bound + F32 * ref.abs()
    bound = bound + (ref.abs() + bound) * half_step(dtype) + tiny(dtype)
    check(y, ref, bound, f"q4_linear {R}x{K}->{N} G={G} {dt}")


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,K,N,G", SHAPES)
def test_rows(R, K, N, G, dt):
    _linear(R, K, N, G, dt, zeros=(R % 2 == 1), bias=(N % 2 == 0))


# Wide enough that a workgroup's block of features is the largest, for every
# block of rows the kernels have.
WIDE_SHAPES = [(1, 200, 13000, 64), (4, 384, 11100, 128), (6, 520, 11000, 32), (16, 264, 2900, 64),
               (20, 392, 11000, 128), (31, 200, 2800, 32), (40, 328, 11000, 64), (64, 136, 5500, 128),
               (90, 264, 11000, 64), (128, 200, 11008, 128), (150, 72, 11008, 32), (256, 392, 8200, 64)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("R,K,N,G", WIDE_SHAPES)
def test_wide_rows(R, K, N, G, dt):
    _linear(R, K, N, G, dt, zeros=True, bias=True, seed=2)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("R,K,N,G", WIDE_SHAPES)
def test_wide_gated_rows(R, K, N, G, dt):
    gen = torch.Generator().manual_seed(4)
    dtype = DTYPES[dt]
    wg, wu = (make_q4(gen, N, K, G, dtype, z, DEV) for z in (False, True))
    x = _x(gen, R, K, dtype)
    (g, dg), (u, du) = (q4_product(x, w, K, G, False) for w in (wg, wu))
    h = sg.q4_gated_ffn(x, *(sg.q4_pack(*w, group_size=G, in_features=K) for w in (wg, wu)))
    check(h, *gated_forward(g, u, dg, du, "silu", dtype), f"wide gated {R}x{K}->{N} G={G} {dt}")


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,K,N,G", TILE_SHAPES)
def test_tiles(R, K, N, G, dt):
    _linear(R, K, N, G, dt, zeros=True, bias=True)
    _linear(R, K, N, G, dt, zeros=False, bias=False, seed=1)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_wide_tiles(dt):
    _linear(3300, 200, 4096, 64, dt, zeros=True, bias=True)


# A little more than a round of 256 x 256 tiles: the rest of the rows or of the
# columns takes smaller ones.
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("R,K,N,G", [(4352, 72, 4400, 32), (2300, 136, 7500, 64), (4100, 40, 4200, 128)])
def test_rest_tiles(R, K, N, G, dt):
    _linear(R, K, N, G, dt, zeros=True, bias=True, seed=12)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("R,K,N,G", [(4200, 72, 2200, 64), (2300, 40, 4000, 128)])
def test_gated_rest_tiles(R, K, N, G, dt):
    gen = torch.Generator().manual_seed(13)
    dtype = DTYPES[dt]
    wg, wu = (make_q4(gen, N, K, G, dtype, z, DEV) for z in (True, False))
    x = _x(gen, R, K, dtype)
    (g, dg), (u, du) = (q4_product(x, w, K, G, True) for w in (wg, wu))
    h = sg.q4_gated_ffn(x, *(sg.q4_pack(*w, group_size=G, in_features=K) for w in (wg, wu)))
    check(h, *gated_forward(g, u, dg, du, "silu", dtype), f"gated rest {R}x{K}->{N} G={G} {dt}")


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
@pytest.mark.parametrize("R,K,N,G", [(1, 256, 64, 128), (7, 136, 43, 32), (40, 520, 96, 64),
                                     (300, 392, 200, 128), (600, 168, 5000, 64)])
def test_gated(R, K, N, G, act, dt):
    gen = torch.Generator().manual_seed(3)
    dtype = DTYPES[dt]
    wg, wu = (make_q4(gen, N, K, G, dtype, z, DEV) for z in (True, False))
    x = _x(gen, R, K, dtype)
    ag, au = (torch.randn(R, N, generator=gen).to(dtype).to(DEV) for _ in range(2))
    pg, pu = (sg.q4_pack(*w, group_size=G, in_features=K) for w in (wg, wu))
    rounded = R > TILE_ROWS and dt != "f32"
    (g, dg), (u, du) = (q4_product(x, w, K, G, rounded) for w in (wg, wu))
    h = sg.q4_gated_ffn(x, pg, pu, act=act)
    check(h, *gated_forward(g, u, dg, du, act, dtype), f"q4_gated_ffn {act} {dt}")
    g, u = g + ag.double().cpu(), u + au.double().cpu()
    dg, du = dg + F32 * g.abs(), du + F32 * u.abs()
    h = sg.q4_gated_ffn(x, pg, pu, act=act, gate_add=ag, up_add=au)
    check(h, *gated_forward(g, u, dg, du, act, dtype), f"q4_gated_ffn {act} {dt} with addends")


def test_integers_are_exact():
    """Small integers with scales of powers of two lose nothing anywhere."""
    gen = torch.Generator().manual_seed(5)
    for R in (1, 20, 300):
        K, N, G = 384, 96, 64
        w = make_q4(gen, N, K, G, torch.float16, True, DEV)
        w = (w[0], torch.full_like(w[1], 0.25), w[2])
        x = torch.randint(-1, 2, (R, K), generator=gen).to(torch.float16).to(DEV)
        y = sg.q4_linear(x, sg.q4_pack(*w, group_size=G))
        q, z, s = q4_parts(w, K, G)
        ref = x.double().cpu() @ (s * (q - z)).t()
        assert torch.equal(y.double().cpu(), ref.to(torch.float16).double())


def test_repeated_calls_agree_and_out_is_written_whole():
    gen = torch.Generator().manual_seed(6)
    w = sg.q4_pack(*make_q4(gen, 100, 512, 128, torch.bfloat16, True, DEV))
    for R in (3, 280):
        x = _x(gen, R, 512, torch.bfloat16)
        out = torch.full((R, 100), float("nan"), dtype=torch.bfloat16, device=DEV)
        y = sg.q4_linear(x, w, out=out)
        assert y is out and torch.equal(y, sg.q4_linear(x, w))


def test_misaligned_x_and_other_rows_untouched():
    gen = torch.Generator().manual_seed(7)
    w4 = make_q4(gen, 72, 256, 64, torch.float16, True, DEV)
    w = sg.q4_pack(*w4, group_size=64)
    for R in (6, 270):
        flat = torch.randn(R * 256 + 1, generator=gen).half().to(DEV)
        x = flat[1:].view(R, 256)  # two bytes off the vector alignment
        y = sg.q4_linear(x, w)
        ref, bound = q4_product(x, w4, 256, 64, R > TILE_ROWS)
        check(y, ref, bound + (ref.abs() + bound) * half_step(torch.float16) + tiny(torch.float16),
              "misaligned x")


def test_bad_rows_stay_alone():
    """Infinities and NaN in one row of x leave the others as they are."""
    gen = torch.Generator().manual_seed(8)
    w = sg.q4_pack(*make_q4(gen, 64, 256, 128, torch.bfloat16, False, DEV))
    for R in (5, 300):
        x = _x(gen, R, 256, torch.bfloat16)
        clean = sg.q4_linear(x, w)
        x[2, 7], x[3, 9] = float("inf"), float("nan")
        y = sg.q4_linear(x, w)
        keep = [i for i in range(R) if i not in (2, 3)]
        assert torch.equal(y[keep], clean[keep])
        assert not bool(torch.isfinite(y[2:4]).any())


def test_empty_batch_and_graph_replay():
    gen = torch.Generator().manual_seed(9)
    w = sg.q4_pack(*make_q4(gen, 48, 128, 64, torch.float16, True, DEV), group_size=64)
    assert sg.q4_linear(torch.empty(0, 128, dtype=torch.float16, device=DEV), w).shape == (0, 48)
    for R in (4, 260):
        x = _x(gen, R, 128, torch.float16)
        out, h = (torch.empty(R, 48, dtype=torch.float16, device=DEV) for _ in range(2))
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            sg.q4_linear(x, w, out=out)
            sg.q4_gated_ffn(x, w, w, out=h)
        for _ in range(3):
            x.copy_(_x(gen, R, 128, torch.float16))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, sg.q4_linear(x, w)) and torch.equal(h, sg.q4_gated_ffn(x, w, w))


def test_runs_on_the_current_stream():
    gen = torch.Generator().manual_seed(10)
    w = sg.q4_pack(*make_q4(gen, 48, 128, 64, torch.float16, True, DEV), group_size=64)
    x = _x(gen, 8, 128, torch.float16)
    want = sg.q4_linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = sg.q4_linear(x * 1, w)
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    gen = torch.Generator().manual_seed(11)
    codes, s, z = make_q4(gen, 32, 128, 64, torch.float16, True, DEV)
    w = sg.q4_pack(codes, s, z, group_size=64)
    x = _x(gen, 2, 128, torch.float16)
    with pytest.raises(ValueError, match="group_size"):
        sg.q4_pack(codes, s, z, group_size=48)
    with pytest.raises(ValueError, match="scales"):
        sg.q4_pack(codes, s, z, group_size=128)
    with pytest.raises(ValueError, match="in_features"):
        sg.q4_pack(codes, s, z, group_size=64, in_features=130)
    with pytest.raises(TypeError, match="codes"):
        sg.q4_pack(codes.int(), s, z, group_size=64)
    with pytest.raises(TypeError, match="float32, float16"):
        sg.q4_pack(codes, s.double(), z, group_size=64)
    with pytest.raises(ValueError, match="input features"):
        sg.q4_linear(x[:, :64].contiguous(), w)
    with pytest.raises(TypeError, match="packed for"):
        sg.q4_linear(x.bfloat16(), w)
    with pytest.raises(ValueError, match="contiguous"):
        sg.q4_linear(_x(gen, 128, 2, torch.float16).t(), w)
    with pytest.raises(ValueError, match="bias"):
        sg.q4_linear(x, w, bias=torch.zeros(31, dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError, match="out"):
        sg.q4_linear(x, w, out=torch.empty(2, 31, dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError, match="act"):
        sg.q4_gated_ffn(x, w, w, act="tanh")
    with pytest.raises(ValueError, match="gate_add"):
        sg.q4_gated_ffn(x, w, w, gate_add=x)
    other = sg.q4_pack(codes, torch.cat([s, s], 1).contiguous(), None, group_size=32)
    with pytest.raises(ValueError, match="disagree"):
        sg.q4_gated_ffn(x, w, other)
