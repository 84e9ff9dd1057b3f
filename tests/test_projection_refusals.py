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
