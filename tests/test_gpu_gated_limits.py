"""gated_ffn at the ends of its activations' ranges."""
import math

import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from proj_helpers import DTYPES, F32, half_step, tiny

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _of_addends(g, u, act, dh):
    """h and dg of the block where x is zero, so that its pre-activations are
    the addends themselves.  g [R, I] decides the kernel by its rows."""
    R, I = g.shape
    x, W = g.new_zeros(R, 64), g.new_zeros(I, 64)
    h = sg.gated_ffn(x, W, W, act, g, u)
    dg, du = sg.gated_ffn_backward(dh, x, W, W, g, u, act, need_dx=False, need_dw=False)[3:]
    return h, dg, du


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R", [2, 40, 300])
def test_gelu_tanh_tail(R, dt):
    """To a relative bound: g sigmoid(2 z), z = k (g + c g^3).  The exponential's
    argument has at most 8 roundings, relative to |2 z| and so to the result; the
    rest of the formula 16.  The derivative is the sum of two such terms."""
    dtype = DTYPES[dt]
    g = torch.linspace(-8, 8, R * 72).to(dtype).view(R, 72)
    one = torch.ones_like(g)
    h, dg, _ = _of_addends(g.to(DEV), one.to(DEV), "gelu_tanh", one.to(DEV))
    g = g.double()
    k = math.sqrt(2 / math.pi)
    z2, slope = 2 * k * (g + 0.044715 * g ** 3), k * (1 + 0.134145 * g * g)
    s, r = torch.sigmoid(z2), torch.sigmoid(-z2)
    rel = F32 * (16 + 8 * z2.abs())
    for got, ref, size in ((h, g * s, (g * s).abs()),
                           (dg, s + 2 * g * s * r * slope, s + (2 * g * s * r * slope).abs())):
        e = size * rel
        bound = e + (ref.abs() + e) * half_step(dtype) + tiny(dtype)
        err = (got.double().cpu() - ref).abs()
        i = int((err / bound).argmax())
        assert bool((err <= bound).all()), (float(g.flatten()[i]), float(got.flatten()[i]), float(ref.flatten()[i]))
