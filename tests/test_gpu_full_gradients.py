"""gated_ffn with full_gradients: nothing between dh and the gradients' own rounding
is held in 16 bits."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from choice_shapes import FFN16, FFN16_SLOW
from exact_helpers import check_exact, exact_block, exact_gated
from proj_helpers import DTYPES, act64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _gradients64(x, Wg, Wu, ag, au, dh, act):
    x, Wg, Wu, ag, au, dh = (t.detach().double() for t in (x, Wg, Wu, ag, au, dh))
    g, u = x @ Wg.t() + ag, x @ Wu.t() + au
    a, d = act64(act, g.cpu())
    a, d = a.to(DEV), d.to(DEV)
    dg, du = dh * u * d, dh * a
    return [a * u, dg @ Wg + du @ Wu, dg.t() @ x, du.t() @ x, dg, du]


def test_the_default_is_full():
    gen = torch.Generator().manual_seed(4)
    x, Wg, Wu, ag, au, dh = exact_block(gen, 90, 72, 104, torch.bfloat16, DEV)
    leaves = [t.requires_grad_() for t in (x, Wg, Wu, ag * 171, au * 171)]
    got = torch.autograd.grad(sg.gated_ffn(x, Wg, Wu, "relu", *leaves[3:]), leaves, dh)
    for a, b in zip(got, _run(leaves, dh, "relu", True)[1:]):
        assert torch.equal(a, b)
    assert not torch.equal(got[0], _run(leaves, dh, "relu", False)[1])


def _run(leaves, dh, act, full):
    h = sg.gated_ffn(*leaves[:3], act, *leaves[3:], full_gradients=full)
    return [h.detach(), *torch.autograd.grad(h, leaves, dh)]


# The root mean square error is that of rounding the result itself, and a twentieth
# more: two parts leave 2^-17 (bf16) or 2^-22 (fp16, until the second part is
# subnormal) of dg and du, and float32 sums of at most 4200 terms 2^-13 at the very most.
# With 16-bit intermediates it is 1.5 to 2 times that.
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("R,H,I", [(40, 264, 200), (300, 520, 1000), (1237, 1000, 2744), (130, 131, 301)])
def test_error_is_the_results_own_rounding(R, H, I, act, dt):
    gen = torch.Generator().manual_seed(R)
    t = lambda *s, k=1.0: (torch.randn(*s, generator=gen) * k).to(DTYPES[dt]).to(DEV).requires_grad_()
    leaves = [t(R, H), t(I, H, k=H ** -0.5), t(I, H, k=H ** -0.5), t(R, I, k=0.3), t(R, I, k=0.3)]
    dh = t(R, I, k=0.5).detach()
    want = _gradients64(*leaves, dh, act)
    rms = lambda e: float(e.square().mean().sqrt())
    for name, got, ref in zip(("h", "dx", "dWg", "dWu", "dg", "du"), _run(leaves, dh, act, True), want):
        own = rms(ref.to(got.dtype).double() - ref)
        assert rms(got.double() - ref) <= 1.05 * own, (name, rms(got.double() - ref) / own)


# Whole numbers that need more than 8 bits in g, u, dg and du: held in bf16 they
# would not give these results.
@pytest.mark.parametrize("dt", ["bf16", "f16"])  # fp16 holds them: the same kernels' sums
@pytest.mark.parametrize("R,H,I", FFN16 + FFN16_SLOW)
def test_exact_where_16_bits_are_not_enough(R, H, I, dt):
    gen = torch.Generator().manual_seed(R + H + I)
    x, Wg, Wu, ag, au, dh = exact_block(gen, R, H, I, DTYPES[dt], DEV)
    ag, au = ag * 171, au * 171  # up to 513: 10 bits with g's own
    leaves = [t.requires_grad_() for t in (x, Wg, Wu, ag, au)]
    got = _run(leaves, dh, "relu", True)
    want = exact_gated(x, Wg, Wu, ag, au, dh, most=1024)
    for name, a, b in zip(("h", "dx", "dWg", "dWu", "dg", "du"), got, want):
        check_exact(a, b, f"{name} of {R}x{H}->{I}")
    some = sg.gated_ffn_backward(dh, x.detach(), Wg.detach(), Wu.detach(), *_kept(leaves), "relu",
                                 need_dx=False)
    assert some[0] is None
    check_exact(some[1], want[2], "dWg without dx")


def _kept(leaves):
    """g and u in float32."""
    x, Wg, Wu, ag, au = (t.detach().double() for t in leaves)
    return [(x @ W.t() + a).float() for W, a in ((Wg, ag), (Wu, au))]


def test_float32_is_the_same_call():
    gen = torch.Generator().manual_seed(1)
    x, Wg, Wu, ag, au, dh = exact_block(gen, 60, 72, 104, torch.float32, DEV)
    leaves = [t.requires_grad_() for t in (x, Wg, Wu, ag, au)]
    for a, b in zip(_run(leaves, dh, "silu", True), _run(leaves, dh, "silu", False)):
        assert torch.equal(a, b)


def test_kept_past_half_precision_and_no_rows():
    x = torch.full((2, 64), 1.0, dtype=torch.float16, device=DEV)
    W = torch.full((8, 64), 152.0, dtype=torch.float16, device=DEV)
    add = torch.full((2, 8), 59904.0,  # g = 69632
                      dtype=torch.float16, device=DEV).requires_grad_()
    h = sg.gated_ffn(x, W, W * 0, "relu", add, torch.ones_like(add) * 2.0 ** -4, full_gradients=True)
    dh = torch.full_like(h, 2.0 ** -4)
    dg, = torch.autograd.grad(h, [add], dh)
    assert float(h.detach().max()) == 4352 and float(dg.max()) == 2.0 ** -8
    up = (torch.ones_like(add) * 2.0 ** -4).detach().requires_grad_()
    h = sg.gated_ffn(x, W, W * 0, "relu", add.detach(), up, full_gradients=True)
    du, = torch.autograd.grad(h, [up], dh)
    assert float(du.max()) == 4352  # 4094 from a g kept in fp16
    e = x[:0].clone().requires_grad_()
    h = sg.gated_ffn(e, W, W.clone().requires_grad_(), full_gradients=True)
    assert torch.autograd.grad(h.sum(), [e])[0].shape == (0, 64)


def test_repeats_and_graph_replay():
    gen = torch.Generator().manual_seed(2)
    x, Wg, Wu, _, _, dh = exact_block(gen, 150, 136, 2056, torch.bfloat16, DEV)
    g, u = (torch.randn(150, 2056, generator=gen).to(DEV) for _ in range(2))
    first = sg.gated_ffn_backward(dh, x, Wg, Wu, g, u)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        res = sg.gated_ffn_backward(dh, x, Wg, Wu, g, u)
    for n in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = sg.gated_ffn_backward(dh, x, Wg, Wu, g, u)
        assert all(torch.equal(a, b) for a, b in zip(res, want))
        assert n or all(torch.equal(a, b) for a, b in zip(res, first))
        g.copy_(torch.randn(g.shape, generator=gen))


def test_refusals():
    gen = torch.Generator().manual_seed(3)
    x, Wg, Wu, _, _, dh = exact_block(gen, 4, 40, 48, torch.float16, DEV)
    with pytest.raises(TypeError, match="u must be"):
        sg.gated_ffn_backward(dh, x, Wg, Wu, dh.float(), dh)  # kept in one type
    with pytest.raises(TypeError, match="g must be"):
        sg.gated_ffn_backward(dh, x, Wg, Wu, dh.bfloat16(), dh.bfloat16())
