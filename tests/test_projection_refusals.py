"""What the projections' calls refuse, on the CPU: nothing is reached but the
check itself."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg


def test_q4_refuses_to_drop_gradients():
    x = torch.zeros(2, 64, requires_grad=True)
    y = torch.zeros(2, 64)
    for call in (lambda: sg.q4_linear(x, None), lambda: sg.q4_linear(y, None, bias=x[0]),
                 lambda: sg.q4_linear(y, None, out=x), lambda: sg.q4_gated_ffn(x, None, None),
                 lambda: sg.q4_gated_ffn(y, None, None, gate_add=x),
                 lambda: sg.q4_gated_ffn(y, None, None, up_add=x)):
        with pytest.raises(RuntimeError, match="has no gradients"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="must be on"):
            call()  # past that check: it refuses the CPU


def test_tangents_are_refused():
    import torch.autograd.forward_ad as fwd
    x, q = torch.zeros(2, 64), torch.zeros(2, 1, 64)
    plan = sg.rope_plan(64, device="cpu")
    pos = torch.zeros(2, dtype=torch.int64)
    with fwd.dual_level():
        d, dq = fwd.make_dual(x, torch.ones_like(x)), fwd.make_dual(q, torch.ones_like(q))
        leaf = fwd.make_dual(x.clone().requires_grad_(), torch.ones_like(x))
        for call in (lambda: sg.q4_linear(d, None), lambda: sg.q4_gated_ffn(x, None, None, gate_add=d),
                     lambda: sg.gated_ffn(d, x, x), lambda: sg.gated_ffn(x, d, x),
                     lambda: sg.gated_ffn(x, x, x, up_add=d), lambda: sg.gated_ffn(leaf, x, x),
                     lambda: sg.rope(dq, None, pos, plan), lambda: sg.rope(q, dq, pos, plan)):
            with pytest.raises(RuntimeError, match="forward-mode"):
                call()
        with pytest.raises(ValueError, match="must be on"):
            sg.gated_ffn(x, x, x)  # no tangent: past that check
