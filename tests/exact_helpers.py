"""Inputs on which the projections' float32 sums lose nothing, so that a lost,
repeated or stale part of a sum shows as a difference.

4-bit weights: x is whole numbers up to 2, scales are 2^-5 (1 + i / 128) with
whole i, so a weight less its zero point times x is a multiple of 2^-12.  Every
partial sum of the sizes used here stays below 2^10 and so within 24 bits, in any
order, biased codes (whole numbers below 2^17) included.  The scaled weight
itself has up to 12 significant bits, more than fp16 (11) and bf16 (8) hold: a
kernel that rounds it first does not give these results.

Gated block: everything is a whole number, g and u of at most 8 bits.
"""
from __future__ import annotations

import torch

from proj_helpers import half_step, make_q4, tiny

F32 = 2.0 ** -24


def exact_q4(gen, N, K, G, dtype, zeros, device):
    codes, scales, z = make_q4(gen, N, K, G, dtype, zeros, "cpu")
    scales = ((1 + torch.randint(0, 128, scales.shape, generator=gen) / 128) * 2.0 ** -5).to(dtype)
    return tuple(None if t is None else t.to(device) for t in (codes, scales, z))


def exact_x(gen, R, K, dtype, device):
    return torch.randint(-2, 3, (R, K), generator=gen).to(dtype).to(device)


def exact_sum(x, w, K, G):
    """x W^T in float64 (no rounding at all), on x's device."""
    codes, s, z = w
    q = torch.stack([codes & 15, codes >> 4], 2).flatten(1)[:, :K].double()
    spread = lambda t: t.double().repeat_interleave(G, 1)[:, :K]
    y = x.double() @ (spread(s) * (q - (spread(z) if z is not None else 8.0))).t()
    assert float(y.abs().max()) < 2 ** 10  # the sums above stay exact
    return y


def check_exact(got, ref, what):
    """got is ref rounded once."""
    want = ref.to(got.dtype)
    assert torch.equal(got, want), \
        f"{what}: {int((got != want).sum())} of {want.numel()} differ, " \
        f"most by {float((got.double() - ref).abs().max()):.3g}"


def check_product(got, g, u, what):
    """got is relu(g) u: one float32 rounding and one to its type."""
    ref = g.clamp(min=0) * u
    bound = ref.abs() * (half_step(got.dtype) * (1 + F32) + F32) + tiny(got.dtype)
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), f"{what}: {int((err > bound).sum())} of {err.numel()} differ"


def exact_block(gen, R, H, I, dtype, device):
    """x, Wg, Wu, gate_add, up_add, dh of whole numbers."""
    t = lambda *s: torch.randint(-1, 2, s, generator=gen).to(dtype).to(device)
    W = lambda: t(I, H) * (torch.rand(I, H, generator=gen) < 0.5).to(dtype).to(device)
    return t(R, H), W(), W(), t(R, I) * 3, t(R, I) * 2, t(R, I)


def exact_gated(x, Wg, Wu, ag, au, dh, most=256):
    """h of relu and the five gradients, before their one rounding."""
    x, Wg, Wu, dh = (t.detach().double() for t in (x, Wg, Wu, dh))
    g, u = x @ Wg.t(), x @ Wu.t()
    if ag is not None:
        g, u = g + ag.detach().double(), u + au.detach().double()
    # 256: g and u are kept in bf16 as they are
    assert float(g.abs().max()) <= most and float(u.abs().max()) <= most
    a = g.clamp(min=0)
    dg, du = dh * u * (g > 0), dh * a
    return [a * u, dg @ Wg + du @ Wu, dg.t() @ x, du.t() @ x, dg, du]
