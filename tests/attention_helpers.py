"""Plain 64-bit forms of the normed rotation, the quantized cache and attention over it, with
elementwise error bounds that count roundings (as in proj_helpers.py)."""
from __future__ import annotations

import math

import torch

from proj_helpers import F32, half_step, tiny

# kind: codes' magnitudes, elements of a group (None: the head), exponents by type
E4M3 = [m / 8 * 2.0 ** -6 for m in range(8)] + [(8 + m) / 8 * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
FORMATS = {"fp8": (E4M3, None, {"f16": (-15, 7), "bf16": (-116, 119), "f32": (-116, 119)}),
           "fp4": (E2M1, 32, {"f16": (-23, 13), "bf16": (-124, 125), "f32": (-124, 125)})}


def kept(x, kind, dt):
    """What a cache keeps of x [..., D], in float64: codes looked up, ties to the even code."""
    grid, group, limits = FORMATS[kind]
    lo, hi = limits[dt]
    grid = torch.tensor(grid, dtype=torch.float64)
    x = x.double().cpu()
    out = torch.empty_like(x)
    for at in range(0, x.shape[-1], group or x.shape[-1]):
        part = x[..., at: at + (group or x.shape[-1])]
        size = part.abs().amax(-1, keepdim=True)
        e = torch.full_like(size, lo)
        for step in range(lo, hi):
            e += (size > grid[-1] * 2.0 ** step).double()
        y = part * torch.exp2(-e)
        between = (grid[1:] + grid[:-1]) / 2
        code = torch.bucketize(y.abs(), between)  # a tie goes down, or to the even code
        tie = y.abs() == between[code.clamp(max=between.numel() - 1)]
        code = (code + (tie & (code % 2 == 1)).long()).clamp(max=grid.numel() - 1)
        val = grid[code] * torch.where(y < 0, -1.0, 1.0) * torch.exp2(e)
        out[..., at: at + part.shape[-1]] = val
    return torch.where(torch.isfinite(x).all(-1, keepdim=True), out, torch.nan)


# -- norm and rotation -------------------------------------------------------------

def _pairs(plan):
    r = plan.rotary_dim
    return (slice(0, r // 2), slice(r // 2, r)) if plan.layout == "half" else (slice(0, r, 2), slice(1, r, 2))


def turned(x, e, pos, plan, inverse=False):
    """(m Rot(t) x, its bound) of x with the bound e.  Cosine and sine carry at most 4 float32
    roundings (argument, function, magnitude), the products and the sum 3; angles are
    float64, off by at most 4 2^-53 of themselves."""
    t = pos.cpu().double()[:, None] * plan.inv_freq.cpu()
    t = -t if inverse else t
    m = plan.magnitude
    c, s = (m * torch.cos(t))[:, None], (m * torch.sin(t))[:, None]
    i, j = _pairs(plan)
    y, b = x.clone(), e.clone()
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    off = (8 * F32 + 4 * 2.0 ** -53 * t.abs()[:, None]) * m
    b[..., i] = b[..., j] = m * (e[..., i] + e[..., j]) + off * (x[..., i].abs() + x[..., j].abs())
    return y, b


def rounded(y, e, dtype):
    return e + (y.abs() + e) * half_step(dtype) + tiny(dtype)


def norm_forward(x, w, pos, plan, eps):
    """(y, bound).  The sum of D squares is off by (D + 1) roundings of itself, its root and
    reciprocal by half of that and 3; two products follow."""
    D, dtype = x.shape[-1], x.dtype
    x = x.double().cpu()
    w = torch.ones(D, dtype=torch.float64) if w is None else w.double().cpu()
    n = x * w / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y, e = turned(n, n.abs() * (D / 2 + 8) * F32, pos, plan)
    return y, rounded(y, e, dtype)


def norm_backward(x, w, dy, pos, plan, eps):
    """((dx, bound), (dw, bound)).  dn = m Rot(-t) dy with its bound e; the mean of w dn x sums D
    terms of 3 roundings each; dx subtracts two products of at most 8 factors."""
    D, dtype = x.shape[-1], x.dtype
    x, dy = x.double().cpu(), dy.double().cpu()
    w = torch.ones(D, dtype=torch.float64) if w is None else w.double().cpu()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    dn, e = turned(dy, torch.zeros_like(dy), pos, plan, inverse=True)
    mean = (w * dn * x).mean(-1, keepdim=True)
    size = (w * dn * x).abs().mean(-1, keepdim=True)
    dx = r * w * dn - x * r ** 3 * mean
    big = r * (w * dn).abs() + x.abs() * r ** 3 * size
    bx = r * w.abs() * e + x.abs() * r ** 3 * ((w * x).abs() * e).mean(-1, keepdim=True) + (2.5 * D + 32) * F32 * big
    terms = dn * x * r
    n = terms.shape[0] * terms.shape[1]
    dw = terms.sum((0, 1))
    bw = ((e * x.abs() * r) + (n + D / 2 + 16) * F32 * (terms.abs() + e * x.abs() * r)).sum((0, 1))
    return (dx, rounded(dx, bx, dtype)), (dw, rounded(dw, bw, dtype))


# -- attention -----------------------------------------------------------------------

def attend(q, k, v, scale):
    """(o, bound, lse, bound) of rows q [N, H, D] over the keys that all of them see, k and v [n, H,
    D] in float64 (n may be 0).

    A score is a float32 sum of D products (of 3 terms for float32 q), scaled: off by d =
    (3 D + 8) roundings of the sum of its terms' magnitudes, and the exponential's argument and
    value by 4 more of the largest score and of 1.  p enters its product in float16
    parts, of 10 fraction bits: half a step is at most 2^-11 of the value, so 2^-11 in one (bfloat16), 2^-22 in two, and what falls below 2^-35 of the
    largest value.  Sums over n keys in any order add n + 16 roundings, twice for
    the quotient."""
    dtype, n = q.dtype, k.shape[0]
    q = q.double().cpu()
    if n == 0:
        z = torch.zeros(q.shape, dtype=torch.float64)
        return z, z, torch.full(q.shape[:2], -math.inf, dtype=torch.float64), z[..., 0]
    kt, vt, qt = (t.transpose(0, 1).contiguous() for t in (k, v, q))
    s = torch.matmul(qt, kt.transpose(1, 2).contiguous()) * scale
    size = torch.matmul(qt.abs(), kt.abs().transpose(1, 2).contiguous()) * scale
    p = torch.softmax(s, -1)
    D = q.shape[-1]
    off = (3 * D + 8) * F32 * size.amax(-1, keepdim=True) + 4 * F32 * (1 + s.abs().amax(-1, keepdim=True))
    part = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22
    o = torch.matmul(p, vt)
    mass = torch.matmul(p, vt.abs())
    bound = mass * (2 * off + part + 2 * (n + 16) * F32) + vt.abs().amax(1, keepdim=True) * n * 2.0 ** -35
    lse = torch.logsumexp(s, -1)
    lse_bound = off[..., 0] + (n + 16) * F32 + 4 * F32 * lse.abs()
    back = lambda t: t.transpose(0, 1)
    return back(o), rounded(back(o), back(bound), dtype), lse.t(), lse_bound.t()
