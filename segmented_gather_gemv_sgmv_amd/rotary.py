"""Rotary positions on q and k.

    plan = rope_plan(128, base=10000.0, layout="half", device="cuda")
    q, k = rope(q, k, positions, plan)             # new tensors
    rope(q, k, positions, plan, out=(q, k))        # in place

q [R, q heads, D] and k [R, k heads, D] may be views of a fused projection's
output (any row and head strides); the first ``rotary_dim`` elements of a
head turn, the rest is copied.  Differentiable (in reverse mode) in q and k.
"""
from __future__ import annotations

import ctypes
import math

from . import _check, _need, _no_tangents, _stream_ptr, _torch, dtype_code, lib

LAYOUTS = {"half": 0, "interleaved": 1}


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling=None):
    """``(inv_freq, magnitude)``: rotary_dim / 2 radians per position (a list
    of floats) and the factor on the rotated elements.

    inv_freq[j] = base^(-2 j / rotary_dim), changed for contexts longer than
    the trained one by ``scaling``, a dict with "kind" and "factor":
      linear    every frequency divided by factor
      ntk       base raised so that the slowest pair slows by factor and the
                fastest keeps its frequency: base * factor^(r / (r - 2))
      by_parts  pairs that turn at least "fast" (32) times within "context"
                positions keep their frequency, those that turn at most
                "slow" (1) times are divided by factor, a linear ramp over
                the pair index between; magnitude = 0.1 ln(factor) + 1 unless
                "magnitude" is given.
    """
    r = int(rotary_dim)
    if r < 2 or r % 2:
        raise ValueError(f"rotary_dim must be even and at least 2, got {rotary_dim}")
    if not base > 0:
        raise ValueError("base must be positive")
    magnitude, kind, factor = 1.0, None, 1.0
    if scaling is not None:
        kind, factor = scaling.get("kind"), float(scaling.get("factor", 0.0))
        if kind not in ("linear", "ntk", "by_parts"):
            raise ValueError(f"scaling kind must be linear, ntk or by_parts, got {kind!r}")
        if not factor > 0:
            raise ValueError("scaling needs a positive factor")
        if kind == "ntk" and r > 2:
            base = base * factor ** (r / (r - 2))
    freq = [base ** (-2.0 * j / r) for j in range(r // 2)]
    if kind == "linear":
        freq = [f / factor for f in freq]
    elif kind == "by_parts":
        context = float(scaling.get("context", 0))
        if not context > 0:
            raise ValueError("by_parts scaling needs the trained context")

        def index(turns):  # (real-valued) element index of the pair turning this often
            return r * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo = max(math.floor(index(float(scaling.get("fast", 32)))), 0)
        hi = min(math.ceil(index(float(scaling.get("slow", 1)))), r - 1)
        width = max(hi - lo, 1e-3)
        ramp = [min(max((j - lo) / width, 0.0), 1.0) for j in range(r // 2)]
        freq = [f * (1 - t) + f / factor * t for f, t in zip(freq, ramp)]
        magnitude = float(scaling.get("magnitude", 0.1 * math.log(factor) + 1.0))
    return freq, magnitude


class RopePlan:
    """Frequencies on the device and the layout of the pairs (rope_plan)."""

    def __init__(self, inv_freq, magnitude, rotary_dim, layout):
        self.inv_freq, self.magnitude = inv_freq, magnitude
        self.rotary_dim, self.layout = rotary_dim, layout
        self.device, self.ptr = inv_freq.device, inv_freq.data_ptr()
        self.interleaved = LAYOUTS[layout]


def rope_plan(rotary_dim: int, base: float = 10000.0, scaling=None, layout: str = "half",
              device="cuda") -> RopePlan:
    """Plan for rope: frequencies as in rope_frequencies, ``layout`` "half"
    (element j pairs with j + rotary_dim / 2) or "interleaved" (2 j, 2 j + 1)."""
    torch = _torch()
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be half or interleaved, got {layout!r}")
    freq, magnitude = rope_frequencies(rotary_dim, base, scaling)
    inv_freq = torch.tensor(freq, dtype=torch.float64, device=device)
    return RopePlan(inv_freq, magnitude, int(rotary_dim), layout)


_Strides = ctypes.c_int64 * 8


def _heads(t, name, dev, dtype):
    """Checks one of q, k and their outputs: place, type, dense last dimension."""
    if not t.is_cuda or t.device != dev:
        raise ValueError(f"{name} must be on {dev if t.is_cuda else 'a GPU'}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows, heads, head_dim], got {tuple(t.shape)}")
    st = t.stride()
    if st[2] != 1 and t.shape[2] > 1 and t.numel():
        raise ValueError(f"{name}'s last dimension must be dense")
    return st


def _one(t, name, o, dev, dtype, R, D):
    """(output, its and t's pointers, strides, heads) of q or k."""
    st = _heads(t, name, dev, dtype)
    shape = t.shape
    if shape[0] != R or shape[2] != D:
        raise ValueError(f"q and k disagree on rows or head_dim: {(R, D)}, {tuple(shape)}")
    if o is None:
        o = t.new_empty(shape)
        so = (shape[1] * D, D)
    else:
        so = _heads(o, "out " + name, dev, dtype)
        if o.shape != shape:
            raise ValueError(f"out {name} must be {tuple(shape)}, got {tuple(o.shape)}")
    return o, o.data_ptr(), t.data_ptr(), (st[0], st[1], so[0], so[1]), shape[1]


_ABSENT = (None, None, None, (0, 0, 0, 0), 0)


def _run(q, k, positions, plan, out, inverse):
    first = q if q is not None else k
    if first is None:
        raise ValueError("q or k must be given")
    dev, dtype = first.device, first.dtype
    if first.dim() != 3:
        raise ValueError(f"q and k must be [rows, heads, head_dim], got {tuple(first.shape)}")
    R, _, D = first.shape
    oq, ok = out if out is not None else (None, None)
    q2, qo, qi, qs, hq = _one(q, "q", oq, dev, dtype, R, D) if q is not None else _ABSENT
    k2, ko, ki, ks, hk = _one(k, "k", ok, dev, dtype, R, D) if k is not None else _ABSENT
    wide = positions.element_size()
    if positions.dtype not in _position_types():
        raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
    _need(positions, "positions", dev, None, 1)
    if positions.shape[0] != R:
        raise ValueError(f"positions must be [{R}], got {tuple(positions.shape)}")
    if plan.device != dev:
        raise ValueError(f"the plan must be on {dev}, got {plan.device}")
    if plan.rotary_dim > D:
        raise ValueError(f"rotary_dim {plan.rotary_dim} exceeds head_dim {D}")
    _check(lib().rope(qo, ko, qi, ki, positions.data_ptr(), wide, plan.ptr, plan.magnitude, R, hq,
                      hk, D, plan.rotary_dim, _Strides(*qs, *ks), plan.interleaved, int(inverse),
                      dtype_code(dtype), _stream_ptr(dev)), "rope")
    return q2, k2


_types = None


def _position_types():
    global _types
    if _types is None:
        _types = (_torch().int64, _torch().int32)
    return _types


_function = None


def _autograd_function():
    """The autograd node (made on first use: this package imports torch late).
    The gradient of a rotation is the rotation back, itself differentiable."""
    global _function
    if _function is None:
        torch = _torch()

        class Rope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, positions, plan, inverse):
                ctx.save_for_backward(positions)
                ctx.plan, ctx.inverse = plan, inverse
                q2, k2 = _run(q, k, positions, plan, None, inverse)
                # What needs no gradient must not ask for one after the turn.
                if k2 is not None and not k.requires_grad:
                    ctx.mark_non_differentiable(k2)
                elif q2 is not None and not q.requires_grad:
                    ctx.mark_non_differentiable(q2)
                return q2, k2

            @staticmethod
            def backward(ctx, dq, dk):
                positions, = ctx.saved_tensors
                want_q, want_k = ctx.needs_input_grad[:2]
                if want_q and dq.stride(2) != 1:
                    dq = dq.contiguous()
                if want_k and dk.stride(2) != 1:
                    dk = dk.contiguous()
                gq, gk = _turn(dq if want_q else None, dk if want_k else None, positions, ctx.plan,
                               not ctx.inverse)
                return gq, gk, None, None, None

        _function = Rope
    return _function


def _turn(q, k, positions, plan, inverse):
    """_run, recorded where gradients are."""
    if _torch().is_grad_enabled() and ((q is not None and q.requires_grad) or
                                       (k is not None and k.requires_grad)):
        return (_function or _autograd_function()).apply(q, k, positions, plan, inverse)
    return _run(q, k, positions, plan, None, inverse)


def rope(q, k, positions, plan: RopePlan, out=None, inverse: bool = False):
    """``(q', k')``: every head's pairs turned by positions[row] * frequency
    and scaled by the plan's magnitude, rounded once.  q or k may be None.
    ``positions`` [R] int32 or int64.  ``out=(q, k)`` works in place (or into
    other tensors, which must not overlap the inputs); ``inverse`` turns back,
    which is what the gradients take."""
    if not isinstance(plan, RopePlan):
        raise TypeError("plan must be a RopePlan (see rope_plan)")
    _no_tangents("rope", q, k)
    if out is None:
        return _turn(q, k, positions, plan, inverse)
    if _torch().is_grad_enabled() and any(t is not None and t.requires_grad for t in (q, k)):
        raise ValueError("out cannot be given where gradients are recorded")
    return _run(q, k, positions, plan, out, inverse)
