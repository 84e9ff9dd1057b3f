"""The gradient of one of gated_ffn's weights alone, the other being frozen."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from exact_helpers import check_exact, exact_block, exact_gated
from proj_helpers import DTYPES

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,H,I", [(40, 72, 104), (300, 264, 1000), (140, 131, 201), (0, 64, 48)])
def test_one_weight(R, H, I, dt, full):
    gen = torch.Generator().manual_seed(R + I)
    x, Wg, Wu, ag, au, dh = exact_block(gen, R, H, I, DTYPES[dt], DEV)
    want = exact_gated(x, Wg, Wu, ag, au, dh) if R else [None, None] + [Wg.double() * 0] * 2
    g, u = (x.double() @ W.double().t() + a.double() for W, a in ((Wg, ag), (Wu, au)))
    kept = torch.float32 if full else x.dtype
    for need, at in (((True, False), 1), ((False, True), 2)):
        got = sg.gated_ffn_backward(dh, x, Wg, Wu, g.to(kept), u.to(kept), "relu", need_dx=False, need_dw=need)
        assert got[0] is None and got[3 - at] is None
        check_exact(got[at], want[at + 1], f"need_dw={need}")
        leaf = (Wg if at == 1 else Wu).clone().requires_grad_()
        W = [leaf, Wu] if at == 1 else [Wg, leaf]
        h = sg.gated_ffn(x, *W, "relu", ag, au, full_gradients=full)
        grad, = torch.autograd.grad(h, [leaf], dh)
        check_exact(grad, want[at + 1], "autograd")


def test_only_one_is_computed():
    """The other gradient's memory is not even asked for."""
    x = torch.randn(64, 1024, device=DEV).half()
    Wg, Wu = (torch.randn(4096, 1024, device=DEV).half() for _ in range(2))
    dh = torch.randn(64, 4096, device=DEV).half()
    peak = {}
    for need in ((True, False), (False, True), True):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        start = torch.cuda.memory_allocated()
        out = sg.gated_ffn_backward(dh, x, Wg, Wu, dh, dh, need_dx=False, need_dw=need)
        peak[need] = torch.cuda.max_memory_allocated() - start
        del out
    weight = Wg.numel() * 2
    assert peak[True] - peak[(True, False)] >= weight and peak[True] - peak[(False, True)] >= weight
