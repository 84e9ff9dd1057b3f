"""gated_ffn and its gradients against their plain 64-bit forms."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from proj_helpers import (CURVE, DTYPES, F32, SLOPE, act64, act_error, check, gated_forward,
                          half_step, plain_product, tiny)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ACTS = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"]

# rows, in, hidden: single tokens, every row class of the streaming kernel,
# tiles of ragged rows, K remainders, sizes no vector fits, K below one step.
SHAPES = [(1, 64, 48), (1, 4096, 96), (5, 1000, 333), (17, 136, 40), (33, 131, 51), (64, 520, 72),
          (65, 256, 128), (100, 200, 136), (130, 333, 77), (200, 24, 264), (70, 8, 8), (300, 640, 392)]


def _inputs(R, H, I, dt, add, seed=0):
    gen = torch.Generator().manual_seed(seed)
    d = DTYPES[dt]
    t = lambda *s, k=1.0: (torch.randn(*s, generator=gen) * k).to(d).to(DEV)
    x, Wg, Wu = t(R, H), t(I, H, k=H ** -0.5), t(I, H, k=H ** -0.5)
    ag, au = (t(R, I, k=0.3), t(R, I, k=0.3)) if add else (None, None)
    return x, Wg, Wu, ag, au, t(R, I, k=0.5)


def _pre(x, Wg, Wu, ag, au):
    """g, u and their bounds."""
    out = []
    for W, a in ((Wg, ag), (Wu, au)):
        v, b = plain_product(x, W)
        if a is not None:
            v = v + a.double().cpu()
            b = b + F32 * v.abs()
        out += [v, b]
    return out


def _check_grads(x, Wg, Wu, ag, au, dh, act, got, what):
    """got: dict of dx, dWg, dWu, dg, du (those computed)."""
    dtype = x.dtype
    u16 = half_step(dtype)
    g, eg, u, eu = _pre(x, Wg, Wu, ag, au)
    eg, eu = (e + (v.abs() + e) * u16 + tiny(dtype) for v, e in ((g, eg), (u, eu)))  # kept rounded
    a, d = act64(act, g)
    h = dh.double().cpu()
    near = (g.abs() <= eg).double() if act == "relu" else 0.0  # the kink: either slope
    ea = SLOPE * eg + act_error(g)
    ed = CURVE * eg + act_error(g) + near
    rdg, rdu = h * u * d, h * a
    edg = h.abs() * ((u.abs() + eu) * ed + d.abs() * eu) + 2 * F32 * rdg.abs()
    edu = h.abs() * ea + F32 * rdu.abs()
    edg = edg + (rdg.abs() + edg) * u16 + tiny(dtype)
    edu = edu + (rdu.abs() + edu) * u16 + tiny(dtype)
    rounded = lambda r, e: e + (r.abs() + e) * u16 + tiny(dtype)
    if "dg" in got:
        check(got["dg"], rdg, edg, what + " dg")
        check(got["du"], rdu, edu, what + " du")
    xd, G, U = x.double().cpu(), Wg.double().cpu(), Wu.double().cpu()
    if "dx" in got:
        n = 2 * G.shape[0] + 8
        ref = rdg @ G + rdu @ U
        e = edg @ G.abs() + edu @ U.abs() + \
            n * F32 * ((rdg.abs() + edg) @ G.abs() + (rdu.abs() + edu) @ U.abs())
        check(got["dx"], ref, rounded(ref, e), what + " dx")
    for name, r, er in (("dWg", rdg, edg), ("dWu", rdu, edu)):
        if name in got:
            ref = r.t() @ xd
            e = er.t() @ xd.abs() + (xd.shape[0] + 8) * F32 * ((r.abs() + er).t() @ xd.abs())
            check(got[name], ref, rounded(ref, e), f"{what} {name}")


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,H,I", SHAPES)
def test_forward(R, H, I, dt):
    for add in (False, True):
        x, Wg, Wu, ag, au, _ = _inputs(R, H, I, dt, add)
        h = sg.gated_ffn(x, Wg, Wu, gate_add=ag, up_add=au)
        g, eg, u, eu = _pre(x, Wg, Wu, ag, au)
        check(h, *gated_forward(g, u, eg, eu, "silu", x.dtype), f"gated_ffn {R}x{H}->{I} {dt}")


# Rows and features enough for tiles in the 16-bit types too: ragged tiles of rows
# and features, K remainders, K below one step.
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,H,I", [(520, 72, 1000), (1000, 520, 520), (130, 24, 4400), (2000, 8, 300),
                                   (700, 200, 904)])
def test_forward_by_tiles(R, H, I, dt):
    x, Wg, Wu, ag, au, _ = _inputs(R, H, I, dt, True, seed=9)
    h = sg.gated_ffn(x, Wg, Wu, gate_add=ag, up_add=au)
    g, eg, u, eu = _pre(x, Wg, Wu, ag, au)
    check(h, *gated_forward(g, u, eg, eu, "silu", x.dtype), f"gated_ffn {R}x{H}->{I} {dt}")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("R", [3, 90])
def test_activations(act, R):
    x, Wg, Wu, ag, au, dh = _inputs(R, 72, 104, "f32", True)
    ag[0, :8] = torch.tensor([0.0, 30.0, -30.0, 90.0, -90.0, 1e4, -1e4, -0.0], device=DEV)
    h = sg.gated_ffn(x, Wg, Wu, act=act, gate_add=ag, up_add=au)
    g, eg, u, eu = _pre(x, Wg, Wu, ag, au)
    check(h, *gated_forward(g, u, eg, eu, act, x.dtype), f"gated_ffn {act}")
    gs, us = g.float().to(DEV), u.float().to(DEV)
    dx, dWg, dWu, dg, du = sg.gated_ffn_backward(dh, x, Wg, Wu, gs, us, act)
    _check_grads(x, Wg, Wu, ag, au, dh, act, dict(dx=dx, dWg=dWg, dWu=dWu, dg=dg, du=du), act)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,H,I", SHAPES)
def test_gradients(R, H, I, dt):
    x, Wg, Wu, ag, au, dh = _inputs(R, H, I, dt, True, seed=1)
    leaves = [t.requires_grad_() for t in (x, Wg, Wu, ag, au)]
    h = sg.gated_ffn(x, Wg, Wu, gate_add=ag, up_add=au)
    grads = torch.autograd.grad(h, leaves, dh)
    with torch.no_grad():
        _check_grads(x, Wg, Wu, ag, au, dh, "silu",
                     dict(zip(("dx", "dWg", "dWu", "dg", "du"), grads)), f"{R}x{H}->{I} {dt}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_wide_tiles(dt):
    """Enough 256 x 256 tiles for every product to take them."""
    x, Wg, Wu, ag, au, dh = _inputs(3100, 4100 // 8 * 8, 2056, dt, False, seed=2)
    x, Wg, Wu = (t.requires_grad_() for t in (x, Wg, Wu))
    h = sg.gated_ffn(x, Wg, Wu, act="gelu_tanh")
    grads = torch.autograd.grad(h, [x, Wg, Wu], dh)
    with torch.no_grad():
        g, eg, u, eu = _pre(x, Wg, Wu, None, None)
        check(h, *gated_forward(g, u, eg, eu, "gelu_tanh", x.dtype), "wide forward")
        _check_grads(x, Wg, Wu, None, None, dh, "gelu_tanh", dict(zip(("dx", "dWg", "dWu"), grads)),
                     "wide " + dt)


# dx of few tiles and a long sum, taken in ranges: whole and ragged tiles, a
# last range that is shorter, sizes no vector fits, more ranges than tile rows.
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,H,I", [(32, 256, 4096), (300, 136, 2008), (90, 333, 1501), (1, 8, 9000),
                                   (257, 1000, 2744)])
def test_sums_in_ranges(R, H, I, dt):
    x, Wg, Wu, ag, au, dh = _inputs(R, H, I, dt, True, seed=7)
    assert sg.lib().gated_ffn_backward_workspace_bytes(R, H, I, sg.dtype_code(x.dtype)) > 0
    leaves = [t.requires_grad_() for t in (x, ag, au)]
    h = sg.gated_ffn(x, Wg, Wu, gate_add=ag, up_add=au)
    grads = torch.autograd.grad(h, leaves, dh, retain_graph=True)
    with torch.no_grad():
        _check_grads(x, Wg, Wu, ag, au, dh, "silu", dict(zip(("dx", "dg", "du"), grads)),
                     f"ranges {R}x{H}->{I} {dt}")
    assert torch.equal(torch.autograd.grad(h, leaves, dh)[0], grads[0])


# Outputs of a little more than a round of 256 x 256 tiles, whose rest takes
# smaller ones: by columns (forward), by rows (the weights' gradients).
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("R,H,I", [(4200, 72, 2200), (70, 4040, 2312), (2050, 40, 8 * 555)])
def test_rest_tiles(R, H, I, dt):
    x, Wg, Wu, ag, au, dh = _inputs(R, H, I, dt, True, seed=8)
    leaves = [t.requires_grad_() for t in (x, Wg, Wu, ag, au)]
    h = sg.gated_ffn(x, Wg, Wu, gate_add=ag, up_add=au)
    grads = torch.autograd.grad(h, leaves, dh)
    with torch.no_grad():
        g, eg, u, eu = _pre(x, Wg, Wu, ag, au)
        check(h, *gated_forward(g, u, eg, eu, "silu", x.dtype), f"rest {R}x{H}->{I} {dt}")
        _check_grads(x, Wg, Wu, ag, au, dh, "silu",
                     dict(zip(("dx", "dWg", "dWu", "dg", "du"), grads)), f"rest {R}x{H}->{I} {dt}")


def test_gradients_against_differences():
    x, Wg, Wu, ag, au, dh = _inputs(6, 40, 24, "f32", True, seed=3)
    leaves = [t.requires_grad_() for t in (x, Wg, Wu, ag, au)]
    for act in ACTS:
        if act == "relu":
            continue  # differences across its kink are not its slope
        grads = torch.autograd.grad(sg.gated_ffn(x, Wg, Wu, act, ag, au), leaves, dh)
        base = [t.detach().double().cpu() for t in leaves]

        def loss(v):
            a, _ = act64(act, v[0] @ v[1].t() + v[3])
            return float((a * (v[0] @ v[2].t() + v[4]) * dh.double().cpu()).sum())

        gen = torch.Generator().manual_seed(4)
        for i, gr in enumerate(grads):
            d = torch.randn(base[i].shape, generator=gen, dtype=torch.float64)
            e = 1e-5
            up, dn = list(base), list(base)
            up[i], dn[i] = base[i] + e * d, base[i] - e * d
            want = (loss(up) - loss(dn)) / (2 * e)
            terms = float((gr.double().cpu() * d).abs().sum())
            # float32 gradients: relative 2^-24 times the longest sum's terms, and
            # the difference quotient's own e^2 and 2^-52 / e parts.
            assert abs(float((gr.double().cpu() * d).sum()) - want) <= 1e-4 * terms + 1e-6, (act, i)


def test_only_what_needs_gradients():
    x, Wg, Wu, ag, au, dh = _inputs(80, 64, 56, "bf16", True)
    leaves = [t.requires_grad_() for t in (x, ag, au)]  # frozen weights
    grads = torch.autograd.grad(sg.gated_ffn(x, Wg, Wu, gate_add=ag, up_add=au), leaves, dh)
    g, _, u, _ = _pre(x.detach(), Wg, Wu, ag.detach(), au.detach())
    dx, dWg, dWu, dg, du = sg.gated_ffn_backward(dh, x.detach(), Wg, Wu, g.bfloat16().to(DEV),
                                                 u.bfloat16().to(DEV), need_dw=False)
    assert dWg is None and dWu is None
    with torch.no_grad():
        _check_grads(x, Wg, Wu, ag, au, dh, "silu", dict(dx=grads[0], dg=grads[1], du=grads[2]),
                     "frozen")
    only = sg.gated_ffn_backward(dh, x.detach(), Wg, Wu, g.bfloat16().to(DEV), u.bfloat16().to(DEV),
                                 need_dx=False)
    assert only[0] is None and only[1] is not None
    # a broadcast upstream gradient (h.sum()) arrives with zero strides
    h = sg.gated_ffn(x, Wg, Wu, gate_add=ag, up_add=au)
    gx, = torch.autograd.grad(h.sum(), [x])
    ones = torch.ones_like(dh)
    gy, = torch.autograd.grad(sg.gated_ffn(x, Wg, Wu, gate_add=ag, up_add=au), [x], ones)
    assert torch.equal(gx, gy)


def test_second_derivative_is_refused():
    x, Wg, Wu, _, _, _ = _inputs(4, 40, 48, "f32", False)
    h = sg.gated_ffn(x.requires_grad_(), Wg, Wu)
    with pytest.raises(RuntimeError, match="once"):
        torch.autograd.grad(h.sum(), [x], create_graph=True)


def test_no_rows():
    x, Wg, Wu, _, _, _ = _inputs(4, 40, 48, "f16", False)
    x0 = x[:0].requires_grad_()
    Wg.requires_grad_(), Wu.requires_grad_()
    h = sg.gated_ffn(x0, Wg, Wu)
    assert h.shape == (0, 48)
    grads = torch.autograd.grad(h, [x0, Wg, Wu], torch.empty(0, 48, dtype=x.dtype, device=DEV))
    assert grads[0].shape == (0, 40)
    assert not bool(grads[1].any()) and not bool(grads[2].any())


def test_misaligned_inputs():
    gen = torch.Generator().manual_seed(5)
    off = lambda *s: torch.randn(torch.Size(s).numel() + 1, generator=gen).half().to(DEV)[1:].view(*s)
    for R in (9, 140):
        x, Wg, Wu, dh = off(R, 64), off(72, 64) * 0.1, off(72, 64), off(R, 72)
        Wu = (torch.cat([Wu.new_zeros(1), Wu.flatten() * 0.1])[1:]).view(72, 64)
        h = sg.gated_ffn(x, Wg, Wu)
        g, eg, u, eu = _pre(x, Wg, Wu, None, None)
        check(h, *gated_forward(g, u, eg, eu, "silu", x.dtype), "misaligned forward")
        dx, dWg, dWu, dg, du = sg.gated_ffn_backward(dh, x, Wg, Wu, g.half().to(DEV),
                                                     u.half().to(DEV))
        _check_grads(x, Wg, Wu, None, None, dh, "silu", dict(dx=dx, dWg=dWg, dWu=dWu, dg=dg, du=du),
                     "misaligned")


def test_repeats_and_graph_replay():
    x, Wg, Wu, _, _, dh = _inputs(150, 136, 200, "bf16", False)
    g, u = (sg.gated_ffn(x, Wg, Wu).float().bfloat16() for _ in range(2))
    assert torch.equal(g, u)
    first = sg.gated_ffn_backward(dh, x, Wg, Wu, g, u)
    again = sg.gated_ffn_backward(dh, x, Wg, Wu, g, u)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    out = torch.empty_like(dh)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sg.gated_ffn(x, Wg, Wu, out=out)
        res = sg.gated_ffn_backward(dh, x, Wg, Wu, g, u)
    gen = torch.Generator().manual_seed(6)
    for _ in range(3):
        x.copy_(torch.randn(x.shape, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, sg.gated_ffn(x, Wg, Wu))
        assert all(torch.equal(a, b)
                   for a, b in zip(res, sg.gated_ffn_backward(dh, x, Wg, Wu, g, u)))


def test_captured_training_pass():
    """Forward and backward through autograd in one graph: replays against eager passes.  No
    eager graph of the captured leaves is alive at the capture."""
    x, Wg, Wu, ag, au, dh = _inputs(120, 136, 2056, "bf16", True, seed=11)
    leaves = [t.requires_grad_() for t in (x, Wg, Wu, ag, au)]
    eager = [t.detach().clone().requires_grad_() for t in leaves]

    def step(v):
        h = sg.gated_ffn(v[0], v[1], v[2], "gelu", v[3], v[4])
        return [h.detach()] + list(torch.autograd.grad(h, v, dh))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(leaves)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(leaves)
    gen = torch.Generator().manual_seed(12)
    for _ in range(3):
        with torch.no_grad():
            for t, e in zip(leaves, eager):
                t.copy_((torch.randn(t.shape, generator=gen) * 0.1).to(t.dtype))
                e.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, step(eager)))


def test_gradients_on_another_stream():
    """dx in ranges, whose workspace is then that stream's, behind other work there."""
    x, Wg, Wu, _, _, dh = _inputs(200, 256, 4096, "f16", False, seed=10)
    g, u = dh * 0.5, dh * 0.25
    want = sg.gated_ffn_backward(dh, x, Wg, Wu, g, u)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a = torch.randn(2048, 2048, device=DEV)
        for _ in range(5):
            a = a @ a * 1e-3
        late = dh.clone() + a[0, 0] * 0
        got = sg.gated_ffn_backward(torch.where(late == late, late, dh), x, Wg, Wu, g, u)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_refusals():
    x, Wg, Wu, ag, _, dh = _inputs(4, 40, 48, "f16", True)
    with pytest.raises(ValueError, match="act"):
        sg.gated_ffn(x, Wg, Wu, act="swish")
    with pytest.raises(ValueError, match="mismatch"):
        sg.gated_ffn(x, Wg, Wu[:40].contiguous())
    with pytest.raises(ValueError, match="mismatch"):
        sg.gated_ffn(x[:, :32].contiguous(), Wg, Wu)
    with pytest.raises(TypeError, match="Wg"):
        sg.gated_ffn(x, Wg.float(), Wu)
    with pytest.raises(ValueError, match="contiguous"):
        sg.gated_ffn(x, Wg.t().contiguous().t(), Wu)
    with pytest.raises(ValueError, match="up_add"):
        sg.gated_ffn(x, Wg, Wu, gate_add=ag, up_add=ag[:3].contiguous())
    with pytest.raises(ValueError, match="on cuda"):
        sg.gated_ffn(x, Wg.cpu(), Wu)
    with pytest.raises(TypeError, match="unsupported dtype"):
        sg.gated_ffn(x.double(), Wg.double(), Wu.double())
    with pytest.raises(ValueError, match="out"):
        sg.gated_ffn(x.requires_grad_(), Wg, Wu, out=torch.empty_like(dh))
    with pytest.raises(ValueError, match="dh"):
        sg.gated_ffn_backward(dh[:2].contiguous(), x.detach(), Wg, Wu, dh, dh)
