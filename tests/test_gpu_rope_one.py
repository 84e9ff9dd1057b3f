"""rope where only one of q and k needs a gradient."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("which", [0, 1])
def test_the_other_output_needs_none(which):
    gen = torch.Generator().manual_seed(1)
    pair = [torch.randn(9, h, 64, generator=gen).to(DEV) for h in (4, 2)]
    pos, plan = torch.arange(9, device=DEV), sg.rope_plan(64, device=DEV)
    want = sg.rope(*pair, pos, plan)
    leaf = pair[which].clone().requires_grad_()
    args = [leaf if i == which else t for i, t in enumerate(pair)]
    out = sg.rope(*args, pos, plan)
    assert all(torch.equal(a.detach(), b) for a, b in zip(out, want))
    assert out[which].requires_grad and not out[1 - which].requires_grad
    sg.rope(out[1 - which], None, pos, plan, out=(out[1 - which], None), inverse=True)  # so this is allowed
    d = torch.randn(pair[which].shape, generator=gen).to(DEV)
    got, = torch.autograd.grad(out[which], [leaf], d, create_graph=True)
    both = [t.clone().requires_grad_() for t in pair]
    ref, = torch.autograd.grad(sg.rope(*both, pos, plan)[which], [both[which]], d)
    assert torch.equal(got, ref)
    # a second derivative through it
    v = torch.randn(pair[which].shape, generator=gen).to(DEV).requires_grad_()
    y = sg.rope(*[v if i == which else t for i, t in enumerate(pair)], pos, plan)[which]
    g, = torch.autograd.grad((y * y).sum(), [v], create_graph=True)
    gg, = torch.autograd.grad(g.sum(), [v])
    assert bool(torch.isfinite(gg).all()) and bool(gg.any())
