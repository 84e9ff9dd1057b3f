"""What the projections' calls refuse, on GPU tensors: gradients and tangents
they would drop, and outputs that overlap their inputs."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import segmented_gather_gemv_sgmv_amd as sg
from proj_helpers import make_q4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def q4():
    gen = torch.Generator().manual_seed(1)
    w = sg.q4_pack(*make_q4(gen, 64, 64, 32, torch.float16, True, DEV), group_size=32)
    x = torch.randn(9, 64, generator=gen).half().to(DEV)
    return x, w


def test_q4_refuses_to_drop_gradients(q4):
    x, w = q4
    leaf, add = x.clone().requires_grad_(), x.clone()
    bias = x[0].clone()
    for call in (lambda: sg.q4_linear(leaf, w), lambda: sg.q4_linear(x, w, bias.clone().requires_grad_()),
                 lambda: sg.q4_gated_ffn(leaf, w, w),
                 lambda: sg.q4_gated_ffn(x, w, w, gate_add=add.clone().requires_grad_()),
                 lambda: sg.q4_gated_ffn(x, w, w, up_add=add.clone().requires_grad_()),
                 lambda: sg.q4_linear(x, w, out=x.clone().requires_grad_())):
        with pytest.raises(RuntimeError, match="gradient"):
            call()
    with torch.no_grad():
        y = sg.q4_linear(leaf, w)
    assert torch.equal(y, sg.q4_linear(leaf.detach(), w)) and not y.requires_grad


def test_tangents_are_refused(q4):
    x, w = q4
    W = torch.randn(64, 64, device=DEV).half()
    q = x.view(9, 1, 64)
    plan, pos = sg.rope_plan(64, device=DEV), torch.arange(9, device=DEV)
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        dq = fwd.make_dual(q, torch.ones_like(q))
        for call in (lambda: sg.q4_linear(dual, w), lambda: sg.q4_gated_ffn(x, w, w, up_add=dual),
                     lambda: sg.gated_ffn(dual, W, W), lambda: sg.gated_ffn(x, W, W, gate_add=dual),
                     lambda: sg.rope(dq, None, pos, plan), lambda: sg.rope(q, dq, pos, plan),
                     lambda: sg.rope(dq, None, pos, plan, out=(torch.empty_like(q), None))):
            with pytest.raises(RuntimeError, match="forward-mode"):
                call()
        sg.q4_linear(x, w), sg.gated_ffn(x, W, W), sg.rope(q, None, pos, plan)  # no tangent: fine
    sg.gated_ffn(x, W, W)


def test_outputs_apart_from_inputs(q4):
    x, w = q4
    W = torch.randn(64, 64, device=DEV).half()
    flat = torch.zeros(3 * 9 * 64, dtype=torch.float16, device=DEV)
    rows = lambda at: flat[at:at + 9 * 64].view(9, 64)
    for out, a in ((rows(0), rows(0)), (rows(64), rows(0)), (rows(0), rows(64))):
        for call in (lambda: sg.q4_linear(a, w, out=out), lambda: sg.q4_gated_ffn(a, w, w, out=out),
                     lambda: sg.gated_ffn(a, W, W, out=out)):
            with pytest.raises(ValueError, match="overlap"):
                call()
    for call in (lambda: sg.q4_linear(x, w, bias=flat[64:128], out=rows(0)),
                 lambda: sg.gated_ffn(x, W, W, out=W[:9]), lambda: sg.gated_ffn(x, W, W.clone(), out=W[5:14]),
                 lambda: sg.q4_gated_ffn(x, w, w, up_add=rows(64), out=rows(0)),
                 lambda: sg.gated_ffn(x, W, W, gate_add=rows(0), out=rows(64))):
        with pytest.raises(ValueError, match="overlap"):
            call()
    # an addend may be the output itself: each element is read where it is written
    add = torch.randn(9, 64, device=DEV).half()
    want = sg.gated_ffn(x, W, W, gate_add=add)
    wantq = sg.q4_gated_ffn(x, w, w, up_add=add)
    a, b = add.clone(), add.clone()
    assert torch.equal(sg.gated_ffn(x, W, W, gate_add=a, out=a), want)
    assert torch.equal(sg.q4_gated_ffn(x, w, w, up_add=b, out=b), wantq)
    sg.q4_linear(rows(0), w, out=rows(9 * 64))  # side by side is apart
