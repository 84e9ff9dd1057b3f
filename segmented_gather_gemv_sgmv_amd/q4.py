"""Projections with 4-bit weights: the quantized base model under 16-bit adapters.

    w = q4_pack(codes, scales, zeros, group_size=128)      # once per weight
    y = q4_linear(x, w, bias)                              # x W^T + bias
    h = q4_gated_ffn(x, w_gate, w_up, act="silu")          # act(x Wg^T) * (x Wu^T)
    lora_apply(y, x, A_stack, B_stack, seg, ids, scale)    # ... and the adapters, as ever

W[n, k] = scales[n, k // group_size] * (code[n, k] - zeros[n, k // group_size]),
zero points 8 where none are given (layouts in include/sgmv.h).  These calls
have no gradients and refuse tensors that would need one; gated_ffn, with plain
weights, has them.
"""
from __future__ import annotations

import ctypes

from . import _check, _need, _no_gradients, _stream_ptr, _torch, dtype_code, lib
from .gated import _act_code, _addends, _output


class _CWeight(ctypes.Structure):
    """sgmv_q4_weight of sgmv.h."""
    _fields_ = [("tiles", ctypes.c_void_p), ("meta", ctypes.c_void_p)]


class Q4Weight:
    """A weight laid out by q4_pack: device arrays and the sizes they were
    made for.  Its dtype is that of the activations it multiplies."""

    def __init__(self, tiles, meta, dtype, out_features, in_features, group_size):
        self.tiles, self.meta, self.dtype = tiles, meta, dtype
        self.out_features, self.in_features = out_features, in_features
        self.group_size = group_size
        self._c = _CWeight(tiles.data_ptr(), meta.data_ptr())
        self._ptr = ctypes.addressof(self._c)

    @property
    def device(self):
        return self.tiles.device


def q4_pack(codes, scales, zeros=None, group_size: int = 128, in_features: int = None) -> Q4Weight:
    """Lays a 4-bit weight out for q4_linear and q4_gated_ffn.

    ``codes`` uint8 [out, ceil(in / 2)] (input feature 2 j in the low half of
    byte j), ``scales`` [out, groups] in the activations' dtype, ``zeros``
    uint8 [out, groups] or None.  ``in_features`` defaults to two per byte
    of a row; give it when it is odd.  ``group_size`` is a multiple of 32."""
    torch = _torch()
    dev = codes.device
    _need(codes, "codes", dev, torch.uint8, 2)
    _need(scales, "scales", dev, None, 2)
    N, nbytes = codes.shape
    K = 2 * nbytes if in_features is None else int(in_features)
    G = int(group_size)
    if K < 1 or (K + 1) // 2 != nbytes:
        raise ValueError(f"codes hold {nbytes} bytes a row, which is not in_features = {K}")
    if G < 32 or G % 32:
        raise ValueError(f"group_size must be a positive multiple of 32, got {G}")
    groups = (K + G - 1) // G
    if tuple(scales.shape) != (N, groups):
        raise ValueError(f"scales must be {(N, groups)}, got {tuple(scales.shape)}")
    dt = dtype_code(scales.dtype)
    if zeros is not None:
        _need(zeros, "zeros", dev, torch.uint8, 2)
        if tuple(zeros.shape) != (N, groups):
            raise ValueError(f"zeros must be {(N, groups)}, got {tuple(zeros.shape)}")
    if N < 1:
        raise ValueError("a weight needs at least one output feature")
    tiles = torch.empty(lib().q4_tiles_bytes(N, K), dtype=torch.uint8, device=dev)
    meta = torch.empty(lib().q4_meta_bytes(N, K, G, dt), dtype=torch.uint8, device=dev)
    _check(lib().q4_pack(tiles.data_ptr(), meta.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                         None if zeros is None else zeros.data_ptr(), N, K, G, dt,
                         _stream_ptr(dev)), "q4_pack")
    return Q4Weight(tiles, meta, scales.dtype, N, K, G)


def _check_weight(w, x, name):
    if not isinstance(w, Q4Weight):
        raise TypeError(f"{name} must be a Q4Weight (see q4_pack)")
    if w.device != x.device:
        raise ValueError(f"{name} must be on {x.device}, got {w.device}")
    if w.dtype != x.dtype:
        raise TypeError(f"{name} was packed for {w.dtype} activations, got {x.dtype}")
    if w.in_features != x.shape[1]:
        raise ValueError(f"{name} takes {w.in_features} input features, got {x.shape[1]}")


def q4_linear(x, w, bias=None, out=None):
    """y = x W^T (+ bias), float32 sums, rounded once.  x [R, in], ``w`` from
    q4_pack, bias [out] or None; ``out`` (optional) receives y [R, out] and must not
    overlap the inputs.  No gradients (see above)."""
    _no_gradients("q4_linear", x, bias, out)
    dev = x.device
    _need(x, "x", dev, None, 2)
    _check_weight(w, x, "w")
    R, N = x.shape[0], w.out_features
    if bias is not None:
        _need(bias, "bias", dev, x.dtype, 1)
        if bias.shape[0] != N:
            raise ValueError(f"bias must be [{N}], got {tuple(bias.shape)}")
    out = _output(out, (R, N), x, x=x, w=w.tiles, w_scales=w.meta, bias=bias)
    _check(lib().q4_linear(out.data_ptr(), x.data_ptr(), w._ptr,
                           None if bias is None else bias.data_ptr(), R, N, w.in_features,
                           w.group_size, dtype_code(x.dtype), _stream_ptr(dev)), "q4_linear")
    return out


def q4_gated_ffn(x, w_gate, w_up, act: str = "silu", gate_add=None, up_add=None, out=None):
    """h = act(x Wg^T + gate_add) * (x Wu^T + up_add) in one kernel, rounded
    once.  x [R, in]; the weights from q4_pack, of one shape and group size;
    the addends [R, out] (or None) are what the rows' adapters contribute
    before the activation; ``out`` (optional) receives h [R, out] and must not overlap
    the inputs (it may be one of the addends itself).  No gradients (see above)."""
    _no_gradients("q4_gated_ffn", x, gate_add, up_add, out)
    dev = x.device
    _need(x, "x", dev, None, 2)
    _check_weight(w_gate, x, "w_gate")
    _check_weight(w_up, x, "w_up")
    if (w_gate.out_features, w_gate.group_size) != (w_up.out_features, w_up.group_size):
        raise ValueError("w_gate and w_up disagree on out_features or group_size")
    R, N = x.shape[0], w_gate.out_features
    code = _act_code(act)
    ga, ua = _addends(gate_add, up_add, (R, N), x)
    out = _output(out, (R, N), x, (gate_add, up_add), x=x, w_gate=w_gate.tiles, w_up=w_up.tiles)
    _check(lib().q4_gated_ffn(out.data_ptr(), x.data_ptr(), w_gate._ptr, w_up._ptr, ga, ua, R, N,
                              w_gate.in_features, w_gate.group_size, code, dtype_code(x.dtype),
                              _stream_ptr(dev)), "q4_gated_ffn")
    return out
