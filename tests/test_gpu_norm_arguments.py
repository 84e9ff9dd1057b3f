"""qk_norm_rope_backward without the gradient of an output."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from attention_helpers import norm_backward
from proj_helpers import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_a_gradient_left_out():
    gen = torch.Generator().manual_seed(90)
    q, k = (torch.randn(5, h, 64, generator=gen).to(DEV) for h in (4, 2))
    w, pos, plan = torch.ones(64, device=DEV), torch.arange(5, device=DEV), sg.rope_plan(64, device=DEV)
    args = (q, k, w, w, pos, plan)
    want = sg.qk_norm_rope_backward(q, k, *args)
    for need, name in (((True, False, False, False), "dq"), ((False, False, True, False), "dq"),
                       ((False, True, False, False), "dk"), ((False, False, False, True), "dk")):
        with pytest.raises(ValueError, match=name + " must be given"):
            sg.qk_norm_rope_backward(None, None, *args, need=need)
    dq, dk, dwq, dwk = sg.qk_norm_rope_backward(q, None, *args, need=(True, False, True, False))
    assert torch.equal(dq, want[0]) and dk is None and dwk is None
    check(dwq, *norm_backward(q, w, q, pos, plan, 1e-6)[1], "dq_weight")  # other workgroups sum it
