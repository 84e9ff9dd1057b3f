"""Plain 64-bit forms of the base projections, the gated block and rotary
positions, with elementwise error bounds, for the tests of their kernels.

Every bound counts roundings.  u is half a step of the tensor's type
relative to the value (finfo.eps / 2); a float32 sum of K terms is off by at
most K 2^-24 of the sum of their magnitudes (to first order, in any order of
summation); one more term or factor adds one more 2^-24.
"""
from __future__ import annotations

import math

import torch

F32 = 2.0 ** -24
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the spacing of the subnormals: what a rounding to zero loses."""
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps / 2


def check(got, ref, bound, what):
    got, ref, bound = got.double().cpu(), ref.cpu(), bound.cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite output"
    err = (got - ref).abs()
    bad = err > bound
    if bool(bad.any()):
        i = int((err - bound).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {err.numel()} out of tolerance; worst "
                             f"{got.flatten()[i]:.8g} against {ref.flatten()[i]:.8g}, error "
                             f"{err.flatten()[i]:.3g} > {bound.flatten()[i]:.3g}")


# -- 4-bit weights ---------------------------------------------------------------

def make_q4(gen, N, K, G, dtype, zeros, device):
    """(codes, scales, zeros) of random codes over the whole range."""
    groups = -(-K // G)
    q = torch.randint(0, 16, (N, K + K % 2), generator=gen, dtype=torch.uint8)
    codes = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    scales = ((0.5 + torch.rand(N, groups, generator=gen)) * (0.2 / math.sqrt(K))).to(dtype)
    z = torch.randint(0, 16, (N, groups), generator=gen, dtype=torch.uint8) if zeros else None
    return tuple(None if t is None else t.to(device) for t in (codes, scales, z))


def q4_parts(w, K, G):
    """Codes [N, K], zero points and scales spread over K, in float64."""
    codes, s, z = (None if t is None else t.cpu() for t in w)
    q = torch.stack([codes & 15, codes >> 4], 2).flatten(1)[:, :K].double()
    spread = lambda t: t.double().repeat_interleave(G, 1)[:, :K]
    zp = spread(z) if z is not None else torch.full_like(q, 8.0)
    return q, zp, spread(s)


def q4_product(x, w, K, G, rounded_weights):
    """(x W^T, its bound before the output's rounding).  Sums run over codes
    biased by 16, x (16 + q) and x (16 + z), each with K + 8 float32 roundings
    (products, scale, zero point, the partial sums' own sums); rounded_weights
    adds one rounding of every scaled weight to x's type."""
    q, z, s = q4_parts(w, K, G)
    xd = x.double().cpu()
    W = s * (q - z)
    ref = xd @ W.t()
    biased = xd.abs() @ (s.abs() * (32 + q + z)).t()
    bound = (K + 8) * F32 * biased
    if rounded_weights:
        bound = bound + xd.abs() @ (W.abs() * half_step(x.dtype) + tiny(x.dtype)).t()
    return ref, bound


# -- activations -------------------------------------------------------------------

def act64(name, g):
    """act(g), act'(g) in float64."""
    if name == "relu":
        return g.clamp(min=0), (g > 0).double()
    if name == "gelu":
        c = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 0.134145 * g * g)
    s = torch.sigmoid(g)
    return (s, s * (1 - s)) if name == "sigmoid" else (g * s, s * (1 + g * (1 - s)))


# Largest |act'| and |act''| of every activation (silu 1.0998 and 0.5, gelu
# 1.1289 and 0.798, its tanh form 1.1290 and 0.81), and float32 roundings in
# the kernel's formulas, whose terms stay below (1 + |g|)^2 ... each.
SLOPE, CURVE = 1.13, 0.82


def act_error(g):
    """Rounding of act and act' in float32: their expressions have at most 32
    roundings (exponential included) on terms no larger than 1 + |g| + |g|^3
    inside the exponential's argument, where the result has decayed."""
    return 32 * F32 * (1 + g.abs())


def gated_forward(g, u, dg, du, act, dtype):
    """(h, bound) from the pre-activations and their error bounds."""
    a, _ = act64(act, g)
    h = a * u
    da = SLOPE * dg + act_error(g)
    e = da * (u.abs() + du) + a.abs() * du + F32 * h.abs()
    return h, e + (h.abs() + e) * half_step(dtype) + tiny(dtype)


def plain_product(x, W):
    xd, Wd = x.double().cpu(), W.double().cpu()
    K = xd.shape[1]
    return xd @ Wd.t(), (K + 8) * F32 * (xd.abs() @ Wd.abs().t())
