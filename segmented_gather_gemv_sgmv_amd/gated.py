"""The gated feed-forward block, both projections in one kernel.

    h = gated_ffn(x, Wg, Wu, act="silu")       # act(x Wg^T + gate_add) * (x Wu^T + up_add)

Differentiable (once, in reverse mode) in x, both weights and both addends;
gated_ffn_backward is the gradient step by itself.  The addends are what the rows' adapters
contribute before the activation (lora_apply_multi on zeros), so that a batch
of many adapters is served, and adapters over a frozen base are trained,
through the same kernel.
"""
from __future__ import annotations

from . import _check, _need, _no_tangents, _stream_ptr, _torch, dtype_code, lib

FULL_GRADIENTS, ONE_WEIGHT = 0x100, 0x200  # options of sgmv.h, OR-ed into the dtype's code

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4}


def _act_code(act) -> int:
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def _output(out, shape, like, addends=(), **inputs):
    """``out`` after its checks, or a new tensor.  A workgroup may write its part of
    ``out`` while others still read the inputs, so it must lie apart from them; an
    addend may be ``out`` itself, each element being read where it is written."""
    if out is None:
        return like.new_empty(shape)
    _need(out, "out", like.device, like.dtype, len(shape))
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must be {tuple(shape)}, got {tuple(out.shape)}")
    lo = out.data_ptr()
    hi = lo + out.numel() * out.element_size()
    others = [*inputs.items()] + [("an addend", a) for a in addends if a is not None and a.data_ptr() != lo]
    for name, t in others:
        if t is not None and lo < t.data_ptr() + t.numel() * t.element_size() and t.data_ptr() < hi:
            raise ValueError(f"out must not overlap {name}")
    return out


def _addends(gate_add, up_add, shape, x):
    """Data pointers of the two addends (None for None)."""
    ptrs = []
    for t, name in ((gate_add, "gate_add"), (up_add, "up_add")):
        if t is not None:
            _need(t, name, x.device, x.dtype, 2)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
        ptrs.append(None if t is None else t.data_ptr())
    return ptrs


def _check_weights(x, Wg, Wu):
    _need(x, "x", x.device, None, 2)
    _need(Wg, "Wg", x.device, x.dtype, 2)
    _need(Wu, "Wu", x.device, x.dtype, 2)
    if Wg.shape != Wu.shape or Wg.shape[1] != x.shape[1]:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, Wg {tuple(Wg.shape)}, "
                         f"Wu {tuple(Wu.shape)}")
    return x.shape[0], x.shape[1], Wg.shape[0]


def _forward(x, Wg, Wu, act, gate_add, up_add, out, kept):
    """(h, g, u); ``kept`` is the type g and u are stored in, None if they are not."""
    R, H, I = _check_weights(x, Wg, Wu)
    code = _act_code(act)
    ga, ua = _addends(gate_add, up_add, (R, I), x)
    out = _output(out, (R, I), x, (gate_add, up_add), x=x, Wg=Wg, Wu=Wu)
    g = u = None
    dtype = dtype_code(x.dtype)
    if kept is not None:
        g, u = x.new_empty((R, I), dtype=kept), x.new_empty((R, I), dtype=kept)
        if kept != x.dtype:
            dtype |= FULL_GRADIENTS
    _check(lib().gated_ffn(out.data_ptr(), None if g is None else g.data_ptr(),
                           None if u is None else u.data_ptr(), x.data_ptr(), Wg.data_ptr(),
                           Wu.data_ptr(), ga, ua, R, H, I, code, dtype,
                           _stream_ptr(x.device)), "gated_ffn")
    return out, g, u


def gated_ffn_backward(dh, x, Wg, Wu, g, u, act: str = "silu", need_dx=True, need_dw=True):
    """Gradients of gated_ffn from dh = dL/dh and the saved g and u (its
    pre-activations, addends included): returns ``(dx, dWg, dWu, dg, du)``,
    dx or the weights' gradients None where not needed; dg and du are also
    the addends' gradients.  ``need_dw`` may be a pair, for Wg and Wu.

    g and u in x's dtype: dg and du are rounded to it too before the products.
    g and u in float32 (x in 16 bits): nothing is rounded but the gradients
    returned, and the products take twice as long."""
    torch = _torch()
    R, H, I = _check_weights(x, Wg, Wu)
    code, dtype = _act_code(act), dtype_code(x.dtype)
    full = g.dtype != x.dtype and g.dtype == torch.float32
    for t, name, kind in ((dh, "dh", x.dtype), (g, "g", g.dtype if full else x.dtype),
                          (u, "u", g.dtype if full else x.dtype)):
        _need(t, name, x.device, kind, 2)
        if tuple(t.shape) != (R, I):
            raise ValueError(f"{name} must be {(R, I)}, got {tuple(t.shape)}")
    need_g, need_u = need_dw if isinstance(need_dw, (tuple, list)) else (need_dw, need_dw)
    dg, du = x.new_empty((R, I)), x.new_empty((R, I))
    dx = x.new_empty((R, H)) if need_dx else None
    dWg = x.new_empty((I, H)) if need_g else None
    dWu = x.new_empty((I, H)) if need_u else None
    if full:
        dtype |= FULL_GRADIENTS
    ptr = lambda t: None if t is None else t.data_ptr()
    ws, ws_bytes = None, 0
    if need_dx or full:
        ws_bytes = lib().gated_ffn_backward_workspace_bytes(R, H, I, dtype)
        if ws_bytes:
            ws = x.new_empty(ws_bytes, dtype=torch.uint8)
    if bool(need_g) != bool(need_u):
        dtype |= ONE_WEIGHT
    _check(lib().gated_ffn_backward(ptr(dx), ptr(dWg), ptr(dWu), dg.data_ptr(), du.data_ptr(),
                                    dh.data_ptr(), x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
                                    g.data_ptr(), u.data_ptr(), R, H, I, code, dtype,
                                    ptr(ws), ws_bytes, _stream_ptr(x.device)),
           "gated_ffn_backward")
    return dx, dWg, dWu, dg, du


_function = None


def _autograd_function():
    """The autograd node (made on first use: this package imports torch late)."""
    global _function
    if _function is None:
        torch = _torch()

        class GatedFFN(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, Wg, Wu, gate_add, up_add, act, full):
                h, g, u = _forward(x, Wg, Wu, act, gate_add, up_add, None,
                                   torch.float32 if full else x.dtype)
                ctx.save_for_backward(x, Wg, Wu, g, u)
                ctx.act = act
                return h

            @staticmethod
            def backward(ctx, dh):
                if torch.is_grad_enabled():  # create_graph: the kernels record nothing
                    raise RuntimeError("gated_ffn can be differentiated once")
                x, Wg, Wu, g, u = ctx.saved_tensors
                want = ctx.needs_input_grad
                dx, dWg, dWu, dg, du = gated_ffn_backward(
                    dh.contiguous(), x, Wg, Wu, g, u, ctx.act, need_dx=want[0], need_dw=want[1:3])
                return (dx, dWg, dWu, dg if want[3] else None, du if want[4] else None, None, None)

        _function = GatedFFN
    return _function


def gated_ffn(x, Wg, Wu, act: str = "silu", gate_add=None, up_add=None, out=None,
              full_gradients: bool = True):
    """h = act(x Wg^T + gate_add) * (x Wu^T + up_add), float32 sums, rounded
    once.  x [R, in], Wg and Wu [hidden, in] (torch's linear layout), addends
    [R, hidden] or None; ``act`` is silu, gelu, gelu_tanh, relu or sigmoid.
    Under autograd the pre-activations are kept in float32 for the backward pass
    and dg and du go through its products in two parts, so that 16-bit gradients
    are off by their own rounding alone.  ``full_gradients=False`` keeps them in
    x's dtype and rounds dg and du to it too, which halves the backward products'
    time and doubles the gradients' error (bf16: 3.1e-3 of their size instead of
    1.7e-3, root mean square).  ``out`` (optional) receives h, is only for
    calls without it, and must not overlap the inputs (it may be one of the
    addends itself).  A backward pass may be captured into a graph once no graph
    that eager calls recorded on the same leaves is alive (the engine would wait
    for their stream inside the capture)."""
    torch = _torch()
    inputs = (x, Wg, Wu, gate_add, up_add)
    _no_tangents("gated_ffn", *inputs)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs):
        if out is not None:
            raise ValueError("out cannot be given where gradients are recorded")
        return _autograd_function().apply(x, Wg, Wu, gate_add, up_add, act, full_gradients)
    return _forward(x, Wg, Wu, act, gate_add, up_add, out, None)[0]
