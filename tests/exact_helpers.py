"""Inputs on which the projections' float32 sums lose nothing, so that a lost,
repeated or stale part of a sum shows as a difference.

4-bit weights: x is whole numbers up to 2, scales are 2^-5 (1 + i / 128) with
whole i, so a weight less its zero point times x is a multiple of 2^-12.  Every
partial sum of the sizes used here stays below 2^10 and so within 24 bits, in any
order, biased codes (whole numbers below 2^17) included.  The scaled weight
itself has up to 12 significant bits, more than fp16 (11) and bf16 (8) hold: a
kernel that rounds it first does not give these results.
"""
from __future__ import annotations

import torch

from proj_helpers import half_step, make_q4, q4_parts, tiny

F32 = 2.0 ** -24


def exact_q4(gen, N, K, G, dtype, zeros, device):
    codes, scales, z = make_q4(gen, N, K, G, dtype, zeros, "cpu")
    scales = (1 + torch.randint(0, 128, scales.shape, generator=gen) / 128).mul(2.0 ** -5).to(dtype)
    return tuple(None if t is None else t.to(device) for t in (codes, scales, z))


def exact_x(gen, R, K, dtype, device):
    return torch.randint(-2, 3, (R, K), generator=gen).to(dtype).to(device)


def exact_sum(x, w, K, G):
    """x W^T in float64 (no rounding at all)."""
    q, z, s = q4_parts(w, K, G)
    y = x.double().cpu() @ (s * (q - z)).t()
    assert float(y.abs().max()) < 2 ** 10  # the sums above stay exact
    return y


def check_exact(got, ref, what):
    """got is ref rounded once."""
    want = ref.to(got.dtype)
    assert torch.equal(got.cpu(), want), \
        f"{what}: {int((got.cpu() != want).sum())} of {want.numel()} differ, " \
        f"most by {float((got.cpu().double() - ref).abs().max()):.3g}"


def check_product(got, g, u, what):
    """got is relu(g) u: one float32 rounding and one to its type."""
    ref = g.clamp(min=0) * u
    bound = ref.abs() * (half_step(got.dtype) * (1 + F32) + F32) + tiny(got.dtype)
    err = (got.double().cpu() - ref).abs()
    assert bool((err <= bound).all()), f"{what}: {int((err > bound).sum())} of {err.numel()} differ"
