"""The normed rotation's cosines and sines, one by one: float32 values of float64 angles, off by steps of
their own size, at far positions and where the sine is small."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _step(y):
    """Distance of float32 values at |y|."""
    return torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -126))) - 23)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("top", [50, 4096, 2 ** 20])
def test_cosines_and_sines(top, layout):
    """x = (1, 0) with eps = 1/2: the mean of the squares is 1/2, the root 1, so the output is (cos, sin)
    itself.  The functions of an argument in float32 are off by up to 2 steps, a correction by what the
    argument lost rounds once more (half a step), and the products with 1 and 0 are exact; the angle is float64, off by
    at most 4 2^-53 of itself (position, frequency, 1 / 2 pi, their products)."""
    rows, pairs = 4096, 8
    gen = torch.Generator().manual_seed(top)
    pos = torch.randint(0, top, (rows,), generator=gen).to(DEV)
    for base in (10000.0, 3.0):
        for j in range(pairs):
            plan = sg.rope_plan(2, layout=layout, device=DEV)
            plan.inv_freq.copy_(torch.tensor([base ** (-j / pairs)], dtype=torch.float64))
            x = torch.tensor([1.0, 0.0], device=DEV).expand(rows, 1, 2)
            got = sg.qk_norm_rope(x, None, None, None, pos, plan, eps=0.5)[0][:, 0].double().cpu()
            t = pos.double().cpu() * plan.inv_freq.cpu()
            want = torch.stack([torch.cos(t), torch.sin(t)], 1)
            bound = 2.5 * _step(want) + 4 * 2.0 ** -53 * t.abs()[:, None]
            err = (got - want).abs()
            assert bool((err <= bound).all()), (base, j, float((err / bound).max()))


def test_gradients_turn_by_the_same_angles():
    """dy = (1, 0) and x = (0, 0) with eps = 1: r = 1 and the second term of dx is 0, so dx = Rot(-t) dy."""
    pos = torch.arange(3000, device=DEV) * 37
    plan = sg.rope_plan(2, device=DEV)
    plan.inv_freq.fill_(0.7310585786300049)
    x = torch.zeros(3000, 1, 2, device=DEV)
    dy = torch.tensor([1.0, 0.0], device=DEV).expand(3000, 1, 2)
    dx = sg.qk_norm_rope_backward(dy, None, x, None, None, None, pos, plan, eps=1.0)[0][:, 0].double().cpu()
    t = pos.double().cpu() * 0.7310585786300049
    want = torch.stack([torch.cos(t), -torch.sin(t)], 1)
    assert bool(((dx - want).abs() <= 2.5 * _step(want) + 4 * 2.0 ** -53 * t[:, None]).all())
