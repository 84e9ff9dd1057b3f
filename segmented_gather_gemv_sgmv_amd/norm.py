"""Norms of queries and keys for each head, with rotary positions in the same pass.

    plan = rope_plan(128, device="cuda")
    q, k = qk_norm_rope(q, k, q_weight, k_weight, positions, plan)      # new tensors
    qk_norm_rope(q, k, q_weight, k_weight, positions, plan, out=(q, k)) # in place

Every head x [D] becomes Rot(x / sqrt(mean(x^2) + eps) * weight), rounded once;
q and k may be views of a fused projection's output, as for rope.  Differentiable
(once, in reverse mode) in q, k and both weights.
"""
from __future__ import annotations

import ctypes

from . import _call_on, _check, _counts, _need, _no_tangents, _stream_ptr, _torch, dtype_code, lib
from .rotary import RopePlan, _ABSENT, _heads, _one, _position_types, _Strides
from .views import apart, repeats

_GradStrides = ctypes.c_int64 * 12


def _weight(w, name, like, D):
    """Pointer of a head's weights (None: ones)."""
    if w is None:
        return None
    _need(w, name, like.device, like.dtype, 1)
    if w.shape[0] != D:
        raise ValueError(f"{name} must be [{D}], got {tuple(w.shape)}")
    return w.data_ptr()


def _common(q, k, q_weight, k_weight, positions, plan):
    """(device, dtype, rows, head_dim) after the checks that both directions share."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("q or k must be given")
    if (q is None and q_weight is not None) or (k is None and k_weight is not None):
        raise ValueError("a weight needs its q or k")
    dev, dtype = first.device, first.dtype
    if first.dim() != 3:
        raise ValueError(f"q and k must be [rows, heads, head_dim], got {tuple(first.shape)}")
    R, H, D = first.shape
    if R > 0x7FFFFFFF or H > 0x7FFFFFFF or D > 0x7FFFFFFF:
        _counts(rows=R, heads=H, head_dim=D)
    if positions.dtype not in _position_types():
        raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
    _need(positions, "positions", dev, None, 1)
    if positions.shape[0] != R:
        raise ValueError(f"positions must be [{R}], got {tuple(positions.shape)}")
    if plan.device != dev:
        raise ValueError(f"the plan must be on {dev}, got {plan.device}")
    if plan.rotary_dim > D:
        raise ValueError(f"rotary_dim {plan.rotary_dim} exceeds head_dim {D}")
    return dev, dtype, R, D


def _own_places(outs, ins, size):
    """Refuses outputs (views, None for new tensors) that share elements with each other, or with an
    input other than as that very view: workgroups read heads when others have written theirs."""
    for i, o in enumerate(outs):
        if o is None:
            continue
        if repeats(o):
            raise ValueError("out must not repeat its own elements")
        other = outs[1 - i]
        if i == 0 and other is not None and not apart(o, other, size):
            raise ValueError("out's q and k must lie apart")
        for j, x in enumerate(ins):  # an output that is an input has been compared as one
            if x is not None and not (o == x if j == i else other == x) and not apart(o, x, size):
                raise ValueError("out must be its input itself or lie apart from the inputs")


def _run(q, k, q_weight, k_weight, positions, plan, eps, out):
    dev, dtype, R, D = _common(q, k, q_weight, k_weight, positions, plan)
    oq, ok = out if out is not None else (None, None)
    q2, qo, qi, qs, hq = _one(q, "q", oq, dev, dtype, R, D) if q is not None else _ABSENT
    k2, ko, ki, ks, hk = _one(k, "k", ok, dev, dtype, R, D) if k is not None else _ABSENT
    if hk > 0x7FFFFFFF:
        _counts(heads=hk)
    wq = _weight(q_weight, "q_weight", q, D)
    wk = _weight(k_weight, "k_weight", k, D)
    if out is not None:
        ins = [None if x is None else (p, R, h, D, s[0], s[1]) for x, p, h, s in ((q, qi, hq, qs), (k, ki, hk, ks))]
        outs = [None if x is None or o is None else (p, R, h, D, s[2], s[3])
                for x, o, p, h, s in ((q, oq, qo, hq, qs), (k, ok, ko, hk, ks))]
        _own_places(outs, ins, dtype.itemsize)
    _check(_call_on(dev, lib().qk_norm_rope, qo, ko, qi, ki, wq, wk, positions.data_ptr(),
                    positions.element_size(), plan.ptr, plan.magnitude, eps, R, hq, hk, D, plan.rotary_dim,
                    _Strides(*qs, *ks), plan.interleaved, dtype_code(dtype), _stream_ptr(dev)), "qk_norm_rope")
    return q2, k2


def _side(x, dy, w, want_x, want_w, name, dev, dtype, R, D):
    """One of q and k in the backward call: (gradients, pointers, strides, heads)."""
    if x is None or not (want_x or want_w):
        return None, None, (None, None, None, None, None), (0,) * 6, 0
    if dy is None:
        raise ValueError(f"d{name} must be given where a gradient of {name} or its weight is wanted")
    sx = _heads(x, name, dev, dtype)
    if dy.shape != x.shape:
        raise ValueError(f"d{name} must be {tuple(x.shape)}, got {tuple(dy.shape)}")
    sg = _heads(dy, "d" + name, dev, dtype)
    H = x.shape[1]
    dx = x.new_empty(x.shape) if want_x else None
    dw = w.new_empty(w.shape) if want_w else None
    ptrs = (None if dx is None else dx.data_ptr(), None if dw is None else dw.data_ptr(), dy.data_ptr(),
            x.data_ptr(), _weight(w, name + "_weight", x, D))
    return dx, dw, ptrs, (sx[0], sx[1], sg[0], sg[1], H * D, D), H


def qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, positions, plan: RopePlan, eps: float = 1e-6,
                          need=(True, True, True, True)):
    """Gradients of qk_norm_rope from those of its outputs: ``(dq, dk, dq_weight,
    dk_weight)``, each None where ``need`` (for q, k, q_weight, k_weight) says so or its
    input is None.  Sums are float32, gradients rounded once, the order of every sum fixed."""
    torch = _torch()
    dev, dtype, R, D = _common(q, k, q_weight, k_weight, positions, plan)
    gq, gqw, pq, sq, hq = _side(q, dq, q_weight, need[0], need[2] and q_weight is not None, "q", dev, dtype, R, D)
    gk, gkw, pk, sk, hk = _side(k, dk, k_weight, need[1], need[3] and k_weight is not None, "k", dev, dtype, R, D)
    if hk > 0x7FFFFFFF:
        _counts(heads=hk)
    ws, ws_bytes = None, 0
    if gqw is not None or gkw is not None:
        ws_bytes = lib().qk_norm_rope_backward_workspace_bytes(R, D, plan.rotary_dim)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _check(_call_on(dev, lib().qk_norm_rope_backward, pq[0], pk[0], pq[1], pk[1], pq[2], pk[2], pq[3], pk[3],
                    pq[4], pk[4], positions.data_ptr(), positions.element_size(), plan.ptr, plan.magnitude,
                    eps, R, hq, hk, D, plan.rotary_dim, _GradStrides(*sq, *sk), plan.interleaved,
                    dtype_code(dtype), None if ws is None else ws.data_ptr(), ws_bytes, _stream_ptr(dev)),
           "qk_norm_rope_backward")
    return gq, gk, gqw, gkw


_function = None


def _autograd_function():
    """The autograd node (made on first use: this package imports torch late)."""
    global _function
    if _function is None:
        torch = _torch()

        class NormRope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, q_weight, k_weight, positions, plan, eps):
                ctx.save_for_backward(q, k, q_weight, k_weight, positions)
                ctx.plan, ctx.eps = plan, eps
                q2, k2 = _run(q, k, q_weight, k_weight, positions, plan, eps, None)
                # What needs no gradient must not ask for one after the turn.
                needs = ctx.needs_input_grad
                if k2 is not None and not (needs[1] or needs[3]):
                    ctx.mark_non_differentiable(k2)
                elif q2 is not None and not (needs[0] or needs[2]):
                    ctx.mark_non_differentiable(q2)
                return q2, k2

            @staticmethod
            def backward(ctx, dq, dk):
                if torch.is_grad_enabled():  # create_graph: the kernels record nothing
                    raise RuntimeError("qk_norm_rope can be differentiated once")
                q, k, q_weight, k_weight, positions = ctx.saved_tensors
                if dq is not None and dq.stride(2) != 1:
                    dq = dq.contiguous()
                if dk is not None and dk.stride(2) != 1:
                    dk = dk.contiguous()
                return (*qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, positions, ctx.plan,
                                               ctx.eps, ctx.needs_input_grad[:4]), None, None, None)

        _function = NormRope
    return _function


def qk_norm_rope(q, k, q_weight, k_weight, positions, plan: RopePlan, eps: float = 1e-6, out=None):
    """``(q', k')``: every head divided by its root mean square (with ``eps`` under the
    root), times its weights, its pairs turned by positions[row] * frequency and scaled
    by the plan's magnitude; float32 in between (squares of elements past 1e19 overflow),
    rounded once.  q [R, q heads, D] and k [R, k heads, D], either may be None; weights [D] in
    their dtype, or None for ones; ``positions`` [R] int32 or int64.  ``out=(q, k)``
    works in place (or into other tensors, which must not overlap the inputs).  A backward pass may be
    captured into a graph once no graph that eager calls recorded on the same leaves is alive."""
    if not isinstance(plan, RopePlan):
        raise TypeError("plan must be a RopePlan (see rope_plan)")
    eps = float(eps)
    if not eps >= 0:
        raise ValueError(f"eps must not be negative, got {eps}")
    inputs = (q, k, q_weight, k_weight)
    _no_tangents("qk_norm_rope", *inputs)
    if _torch().is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs):
        if out is not None:
            raise ValueError("out cannot be given where gradients are recorded")
        return (_function or _autograd_function()).apply(q, k, q_weight, k_weight, positions, plan, eps)
    return _run(q, k, q_weight, k_weight, positions, plan, eps, out)
