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


def test_outputs_apart_from_inputs(monkeypatch):
    """The check itself, on CPU tensors (the GPU's calls make it too)."""
    from segmented_gather_gemv_sgmv_amd import gated
    monkeypatch.setattr(gated, "_need", lambda *a: None)
    flat = torch.zeros(64)
    at = lambda i: flat[i:i + 16].view(4, 4)
    for i in (0, 1, 15):
        for a, b in ((0, i), (i, 0)):
            with pytest.raises(ValueError, match="overlap x"):
                gated._output(at(a), (4, 4), flat, x=at(b))
    out = at(16)
    assert gated._output(out, (4, 4), flat, (out, None), x=at(0), w=at(32), bias=None) is out
    for i in (15, 17):
        with pytest.raises(ValueError, match="overlap an addend"):
            gated._output(out, (4, 4), flat, (None, at(i)), x=at(32))
    none = flat[:0].view(0, 4)
    assert gated._output(none, (0, 4), flat, x=at(0)) is none
