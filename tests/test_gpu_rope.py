"""rope against its plain 64-bit form."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from proj_helpers import DTYPES, F32, check, half_step, tiny

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _reference(x, pos, plan, inverse=False):
    """(rotated, bound).  The kernel's cosine and sine carry at most 4 float32
    roundings (argument, function, magnitude), the products and the sum 3;
    angles are float64, off by at most 4 2^-53 of themselves."""
    x = x.double().cpu()
    f = plan.inv_freq.cpu()
    t = pos.cpu().double()[:, None] * f[None, :]
    if inverse:
        t = -t
    m, r = plan.magnitude, plan.rotary_dim
    c, s = (m * torch.cos(t))[:, None], (m * torch.sin(t))[:, None]
    i, j = (slice(0, r // 2), slice(r // 2, r)) if plan.layout == "half" else \
        (slice(0, r, 2), slice(1, r, 2))
    y, e = x.clone(), torch.zeros_like(x)
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    off = 8 * F32 * m + 4 * 2.0 ** -53 * t.abs()[:, None] * m
    e[..., i] = e[..., j] = off * (a.abs() + b.abs())
    return y, e + (y.abs() + e) * half_step_of(x, e)


def half_step_of(x, e):
    return e.new_tensor(_reference.u) * (e > 0)


def _check(got, x, pos, plan, what, inverse=False):
    _reference.u = half_step(got.dtype)
    ref, bound = _reference(x, pos, plan, inverse)
    r = plan.rotary_dim
    bound[..., :r] += tiny(got.dtype)
    check(got, ref, bound, what)
    assert torch.equal(got[..., r:], x[..., r:]), f"{what}: elements past rotary_dim"


# rows, q heads, k heads, head_dim, rotary_dim
SHAPES = [(1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (7, 4, 2, 80, 32), (33, 3, 1, 96, 50),
          (5, 2, 2, 10, 6), (64, 32, 32, 128, 64), (300, 5, 5, 72, 72), (3, 7, 1, 256, 256),
          (2, 1, 3, 2, 2), (9, 2, 1, 33, 32), (2, 1, 1, 1024, 1024)]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("R,Hq,Hk,D,rot", SHAPES)
def test_forward_and_gradients(R, Hq, Hk, D, rot, layout, dt):
    gen = torch.Generator().manual_seed(R + D)
    qkv = torch.randn(R, Hq + 2 * Hk, D, generator=gen).to(DTYPES[dt]).to(DEV)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]  # views of the fused projection
    pos = torch.randint(0, 5000, (R,), generator=gen).to(DEV)
    plan = sg.rope_plan(rot, layout=layout, device=DEV)
    q2, k2 = sg.rope(q, k, pos, plan)
    _check(q2, q, pos, plan, "q")
    _check(k2, k, pos, plan, "k")
    ql, kl = q.detach().requires_grad_(), k.detach().requires_grad_()
    dq, dk = (torch.randn(t.shape, generator=gen).to(t.dtype).to(DEV) for t in (q, k))
    gq, gk = torch.autograd.grad(sg.rope(ql, kl, pos, plan), [ql, kl], [dq, dk])
    _check(gq, dq, pos, plan, "dq", inverse=True)
    _check(gk, dk, pos, plan, "dk", inverse=True)


@pytest.mark.parametrize("scaling", [None, dict(kind="linear", factor=4.0),
                                     dict(kind="ntk", factor=8.0),
                                     dict(kind="by_parts", factor=16.0, context=4096),
                                     dict(kind="by_parts", factor=2.0, context=2048, magnitude=0.5)])
def test_far_positions_and_scaling(scaling):
    gen = torch.Generator().manual_seed(1)
    plan = sg.rope_plan(128, base=500000.0, scaling=scaling, device=DEV)
    q = torch.randn(40, 2, 128, generator=gen).to(DEV)
    pos = torch.cat([torch.tensor([0, 1, 2 ** 20, 2 ** 31 - 1]),
                     torch.randint(0, 10 ** 6, (36,), generator=gen)]).to(DEV)
    for p in (pos, pos.int()):
        out, none = sg.rope(q, None, p, plan)
        assert none is None
        _check(out, q, p, plan, f"{scaling}")
    far = torch.full((40,), 2 ** 40, device=DEV)  # past 32 bits
    _check(sg.rope(q, None, far, plan)[0], q, far, plan, "far")


def test_frequencies():
    f, m = sg.rope_frequencies(8, base=16.0)
    assert f == [1.0, 0.5, 0.25, 0.125] and m == 1.0
    assert sg.rope_frequencies(8, 16.0, dict(kind="linear", factor=2.0))[0] == [0.5, 0.25, 0.125,
                                                                                  0.0625]
    n, _ = sg.rope_frequencies(8, 16.0, dict(kind="ntk", factor=8.0))
    assert n[0] == 1.0 and abs(n[-1] - 0.125 / 8.0) < 1e-15
    p, m = sg.rope_frequencies(64, 10000.0, dict(kind="by_parts", factor=4.0, context=2048))
    g, _ = sg.rope_frequencies(64, 10000.0)
    assert p[0] == g[0] and abs(p[-1] - g[-1] / 4) < 1e-18 and m > 1.1
    assert all(a >= b for a, b in zip(p, p[1:]))


def test_in_place_on_views_and_back():
    gen = torch.Generator().manual_seed(2)
    for dt in DTYPES.values():
        qkv = torch.randn(20, 12, 64, generator=gen).to(dt).to(DEV)
        keep = qkv.clone()
        q, k = qkv[:, :8], qkv[:, 8:10]
        pos = torch.arange(20, device=DEV)
        plan = sg.rope_plan(48, device=DEV)
        wq, wk = sg.rope(q, k, pos, plan)
        rq, rk = sg.rope(q, k, pos, plan, out=(q, k))
        assert rq is q and rk is k
        assert torch.equal(q, wq) and torch.equal(k, wk) and torch.equal(qkv[:, 10:], keep[:, 10:])
        # Turning back undoes it up to the roundings of both ways.
        sg.rope(q, k, pos, plan, out=(q, k), inverse=True)
        bound = 4 * half_step(dt) * (keep.abs().double().amax() * 2)
        assert float((qkv.double() - keep.double()).abs().max()) <= float(bound)


def test_strides_and_alignment():
    """Heads innermost in memory, rows apart, addresses off the vectors."""
    gen = torch.Generator().manual_seed(3)
    plan = sg.rope_plan(64, device=DEV)
    pos = torch.randint(0, 999, (11,), generator=gen).to(DEV)
    base = torch.randn(5, 11, 64, generator=gen).half().to(DEV)
    x = base.transpose(0, 1)  # [11, 5, 64], head stride above the row stride
    _check(sg.rope(x, None, pos, plan)[0], x, pos, plan, "transposed")
    off = torch.randn(11 * 3 * 64 + 3, generator=gen).half().to(DEV)[3:].view(11, 3, 64)
    _check(sg.rope(None, off, pos, plan)[1], off, pos, plan, "misaligned")
    wide = torch.randn(11, 3, 70, generator=gen).half().to(DEV)[..., 1:65]
    _check(sg.rope(wide, off, pos, plan)[0], wide, pos, plan, "inner slice")
    one = torch.randn(1, 1, 64, generator=gen).half().to(DEV).expand(11, 4, 64)  # broadcast input
    _check(sg.rope(one, None, pos, plan)[0], one, pos, plan, "broadcast")
    leaf = off.clone().requires_grad_()
    got, = torch.autograd.grad(sg.rope(leaf, None, pos, plan)[0].sum(), [leaf])
    _check(got, torch.ones_like(off), pos, plan, "gradient of a sum", inverse=True)


def test_negative_positions_special_values_empty():
    plan = sg.rope_plan(8, device=DEV)
    x = torch.zeros(3, 1, 16, device=DEV)
    x[0, 0, 0], x[1, 0, 3], x[2, 0, 12] = float("inf"), float("nan"), float("-inf")
    y = sg.rope(x, None, torch.tensor([-5, 0, 3], device=DEV), plan)[0]
    assert not bool(torch.isfinite(y[0, 0, [0, 4]]).any())
    assert float(y[2, 0, 12]) == float("-inf") and bool(torch.isfinite(y[2, 0, :8]).all())
    assert bool(torch.isfinite(y[1, 0, [0, 1, 2, 4, 5, 6]]).all())
    e = sg.rope(x[:0], x[:0, :0], torch.zeros(0, dtype=torch.int64, device=DEV), plan)
    assert e[0].shape == (0, 1, 16) and e[1].shape == (0, 0, 16)


def test_graph_replay_and_stream():
    gen = torch.Generator().manual_seed(4)
    plan = sg.rope_plan(64, device=DEV)
    q = torch.randn(30, 4, 64, generator=gen).half().to(DEV)
    pos = torch.arange(30, device=DEV)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sg.rope(q, None, pos, plan, out=(out, None))
    for n in range(3):
        pos.add_(n + 1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, sg.rope(q, None, pos, plan)[0])


def test_refusals():
    plan = sg.rope_plan(64, device=DEV)
    q = torch.zeros(4, 2, 64, device=DEV)
    pos = torch.arange(4, device=DEV)
    with pytest.raises(TypeError, match="plan"):
        sg.rope(q, None, pos, 10000.0)
    with pytest.raises(ValueError, match="must be given"):
        sg.rope(None, None, pos, plan)
    with pytest.raises(ValueError, match="exceeds"):
        sg.rope(q[..., :32], None, pos, plan)
    with pytest.raises(ValueError, match="dense"):
        sg.rope(q.transpose(1, 2), None, pos, plan)
    with pytest.raises(ValueError, match="positions"):
        sg.rope(q, None, pos[:3].contiguous(), plan)
    with pytest.raises(TypeError, match="int32 or int64"):
        sg.rope(q, None, pos.float(), plan)
    with pytest.raises(ValueError, match="disagree"):
        sg.rope(q, q[:3], pos, plan)
    with pytest.raises(TypeError, match="k must be"):
        sg.rope(q, q.half(), pos, plan)
    with pytest.raises(ValueError, match="out q"):
        sg.rope(q, None, pos, plan, out=(q[:, :1], None))
    with pytest.raises(ValueError, match="rows, heads"):
        sg.rope(q[0], None, pos, plan)
    with pytest.raises(ValueError, match="recorded"):
        sg.rope(q.clone().requires_grad_(), None, pos, plan, out=(torch.empty_like(q), None))


def test_second_derivative():
    """<rope(q), rope(q)> has the gradient 2 m^2 q on turned elements, 2 q on
    the others; its own derivative is that factor again."""
    gen = torch.Generator().manual_seed(5)
    plan = sg.rope_plan(32, scaling=dict(kind="by_parts", factor=4.0, context=1024), device=DEV)
    q = torch.randn(6, 2, 48, generator=gen).to(DEV).requires_grad_()
    pos = torch.arange(6, device=DEV)
    out, _ = sg.rope(q, None, pos, plan)
    g, = torch.autograd.grad((out * out).sum(), [q], create_graph=True)
    v = torch.randn(q.shape, generator=gen).to(DEV)
    gg, = torch.autograd.grad(g, [q], v)
    factor = torch.full((48,), 2.0, dtype=torch.float64)
    factor[:32] *= plan.magnitude ** 2
    # two rotations of float32 pairs each way: 4 x 8 roundings of the pair's size
    want = v.double().cpu() * factor
    size = v.double().cpu().abs().amax(-1, keepdim=True) * factor.max() * 2
    check(gg, want, 32 * F32 * size.expand_as(want), "second derivative")
