"""gated_ffn at the ends of its activations' ranges: tails, masks of the
lowest value and of minus infinity, pre-activations past the type's largest."""
import math

import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from proj_helpers import DTYPES, F32, act64, half_step, tiny

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ACTS = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"]


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


def _block(R, H, I, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    t = lambda *s, k=1.0: (torch.randn(*s, generator=gen) * k).to(dtype).to(DEV)
    return t(R, H), t(I, H, k=H ** -0.5), t(I, H, k=H ** -0.5), t(R, I, k=0.3), t(R, I, k=0.3), t(R, I, k=0.5)


# A mask of the type's lowest value or of minus infinity in gate_add takes a hidden
# unit out of a row: it adds nothing to h and to the gradients, in rows that keep
# nothing too.  Their other units are those of the unmasked block, bit for bit.
@pytest.mark.parametrize("low", ["lowest", "infinity"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R", [3, 50, 400])
def test_masked_units(R, dt, act, low):
    dtype = DTYPES[dt]
    x, Wg, Wu, ag, au, dh = _block(R, 72, 104, dtype, 1)
    mask = torch.rand(R, 104, generator=torch.Generator().manual_seed(2)) < 0.5
    mask[0], mask[1] = True, False
    mask = mask.to(DEV)
    value = torch.finfo(dtype).min if low == "lowest" else -math.inf
    leaves = [t.requires_grad_() for t in (x, ag.masked_fill(mask, value), au)]
    h = sg.gated_ffn(x, Wg, Wu, act, leaves[1], leaves[2])
    dx, dg, du = torch.autograd.grad(h, leaves, dh)
    free = [t.detach().clone().requires_grad_() for t in (x, ag, au)]
    hf = sg.gated_ffn(free[0], Wg, Wu, act, free[1], free[2])
    _, dgf, duf = torch.autograd.grad(hf, free, dh)
    for name, got, want in (("h", h, hf), ("dg", dg, dgf), ("du", du, duf)):
        assert not bool(got[mask].any()), f"{name} of masked units"
        assert torch.equal(got[~mask], want[~mask]), f"{name} of the others"
    assert bool(torch.isfinite(dx).all()) and not bool(dx[0].any())


@pytest.mark.parametrize("act", ACTS)
def test_limits_of_the_derivative(act):
    """Where the cubes and squares of g overflow float32, and at infinities."""
    big = [2.0 ** k for k in range(0, 128, 3)] + [3.4e38, math.inf]
    g = torch.tensor([[v * s for v in big for s in (1, -1)]]).expand(3, -1).contiguous()
    one = torch.ones_like(g)
    _, dg, du = _of_addends(g.to(DEV), one.to(DEV), act, one.to(DEV))
    a, d = act64(act, g.double().clamp(-1e3, 1e3))  # act' is at its limits beyond
    want = torch.where(g.abs() > 1e3, g.double().clamp(min=0) if act != "sigmoid" else a, a)
    for got, ref, size in ((dg, d, 1.2), (du, want, 1.0)):
        got = got.double().cpu()
        assert not bool(torch.isnan(got).any())
        fin = torch.isfinite(ref)
        assert torch.equal(got[~fin], ref[~fin])
        assert bool(((got - ref).abs()[fin] <= 64 * F32 * (size + ref.abs()[fin])).all())
    nan = torch.full((1, 8), math.nan, device=DEV)
    h, dg, du = _of_addends(nan, torch.ones_like(nan), act, torch.ones_like(nan))
    assert bool(torch.isnan(h).all()) and bool(torch.isnan(du).all())


@pytest.mark.parametrize("R", [2, 30, 300])
def test_pre_activations_past_half_precision(R):
    """g and u of 70000: kept as the largest finite value, so no gradient is
    infinity times zero.  Where the loss does not depend on h, all are zero."""
    x = torch.ones(R, 64, dtype=torch.float16, device=DEV)
    W = torch.full((80, 64), 156.25, dtype=torch.float16, device=DEV)  # x W^T = 10000
    add = torch.full((R, 80), 60000.0, dtype=torch.float16, device=DEV)
    leaves = [x.requires_grad_(), add.clone().requires_grad_(), add.clone().requires_grad_()]
    for act, sign in (("silu", 1), ("sigmoid", 1), ("relu", -1)):
        h = sg.gated_ffn(leaves[0], sign * W, W, act, sign * leaves[1], leaves[2])
        grads = torch.autograd.grad(h, leaves, torch.zeros_like(h))
        assert not any(bool(g.any()) for g in grads), act  # a NaN counts as set
    g = torch.tensor([[70000.0]], device=DEV)  # in float32 nothing is lost
    one = torch.ones_like(g)
    h = sg.gated_ffn(one, g, one, "relu")
    assert float(h) == 70000.0
