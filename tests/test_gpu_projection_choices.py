"""Every kernel of the projections, the gated block and rope, at shapes that reach it
(choice_shapes.py), on inputs whose sums are exact: results are compared for
equality, so a lost or repeated part of a sum of any length is seen."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from choice_shapes import FFN16, FFN16_SLOW, FFN32, Q4_FEW, Q4_FEW_K, Q4_SLOW, Q4_TILES, ROPE
from exact_helpers import (check_exact, check_product, exact_block, exact_gated, exact_q4, exact_sum,
                           exact_x)
from proj_helpers import DTYPES
from test_gpu_rope import _check as check_rope

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _q4(R, K, N, G, dt):
    gen = torch.Generator().manual_seed(R + K + N)
    dtype = DTYPES[dt]
    wg, wu = (exact_q4(gen, N, K, G, dtype, z, DEV) for z in (True, False))
    x = exact_x(gen, R, K, dtype, DEV)
    add = torch.randint(-4, 5, (N,), generator=gen).to(dtype).to(DEV)
    pg, pu = (sg.q4_pack(*w, group_size=G, in_features=K) for w in (wg, wu))
    g, u = (exact_sum(x, w, K, G) for w in (wg, wu))
    what = f"{R}x{K}->{N} G={G} {dt}"
    check_exact(sg.q4_linear(x, pg), g, "q4_linear " + what)
    check_exact(sg.q4_linear(x, pu, bias=add), u + add.double(), "q4_linear, bias " + what)
    check_product(sg.q4_gated_ffn(x, pg, pu, "relu"), g, u, "q4_gated_ffn " + what)
    rows = add.expand(R, N).contiguous()
    check_product(sg.q4_gated_ffn(x, pg, pu, "relu", rows, rows), g + add.double(), u + add.double(),
                  "q4_gated_ffn, addends " + what)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("R,N", Q4_FEW)
def test_q4_few_rows(R, N, G, dt):
    _q4(R, Q4_FEW_K, N, G, dt)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("R,K,N", Q4_TILES)
def test_q4_tiles(R, K, N, G, dt):
    _q4(R, K, N, G, dt)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("R,K,N", Q4_SLOW)
def test_q4_register_path(R, K, N, G, dt):
    _q4(R, K, N, G, dt)


def _block(R, H, I, dt):
    gen = torch.Generator().manual_seed(R + H + I)
    x, Wg, Wu, ag, au, dh = exact_block(gen, R, H, I, DTYPES[dt], DEV)
    leaves = [t.requires_grad_() for t in (x, Wg, Wu, ag, au)]
    h = sg.gated_ffn(x, Wg, Wu, "relu", ag, au, full_gradients=False)  # True: test_gpu_full_gradients.py
    got = [h.detach(), *torch.autograd.grad(h, leaves, dh)]
    want = exact_gated(x, Wg, Wu, ag, au, dh)
    for name, a, b in zip(("h", "dx", "dWg", "dWu", "dg", "du"), got, want):
        check_exact(a, b, f"{name} of {R}x{H}->{I} {dt}")
    with torch.no_grad():
        check_exact(sg.gated_ffn(x, Wg, Wu, "relu"), exact_gated(x, Wg, Wu, None, None, dh)[0],
                    f"h without addends of {R}x{H}->{I} {dt}")


# A row's result does not depend on the rows beside it, whichever kernels they take: on
# these inputs, bit for bit.
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_q4_rows_are_the_same_in_any_batch(dt):
    gen = torch.Generator().manual_seed(3)
    dtype = DTYPES[dt]
    w = sg.q4_pack(*exact_q4(gen, 9000, 1000, 64, dtype, True, DEV), group_size=64)
    x = exact_x(gen, 700, 1000, dtype, DEV)
    y = sg.q4_linear(x, w)
    for rows in (1, 4, 30, 100, 256, 257, 300):
        assert torch.equal(sg.q4_linear(x[:rows], w), y[:rows]), rows


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("R,H,I", FFN16 + FFN16_SLOW)
def test_gated_block(R, H, I, dt):
    _block(R, H, I, dt)


@pytest.mark.parametrize("R,H,I", FFN32)
def test_gated_block_float32(R, H, I):
    _block(R, H, I, "f32")


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("R,Hq,Hk,D,rot", ROPE)
def test_rope(R, Hq, Hk, D, rot, layout, dt):
    gen = torch.Generator().manual_seed(R)
    qkv = torch.randn(R, Hq + 2 * Hk, D, generator=gen).to(DTYPES[dt]).to(DEV)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    pos = torch.randint(0, 9000, (R,), generator=gen).to(DEV)
    plan = sg.rope_plan(rot, layout=layout, device=DEV)
    ql, kl = q.detach().requires_grad_(), k.detach().requires_grad_()
    out = sg.rope(ql, kl, pos, plan)
    for got, x, name in zip(out, (q, k), "qk"):
        check_rope(got.detach(), x, pos, plan, name)
    d = [torch.randn(t.shape, generator=gen).to(t.dtype).to(DEV) for t in (q, k)]
    for got, x, name in zip(torch.autograd.grad(out, [ql, kl], d), d, ("dq", "dk")):
        check_rope(got, x, pos, plan, name, inverse=True)
    want = [t.detach().clone() for t in out]
    sg.rope(q, k, pos, plan, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
