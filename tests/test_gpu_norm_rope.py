"""qk_norm_rope and its gradients against the plain 64-bit form."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from attention_helpers import norm_backward, norm_forward
from proj_helpers import DTYPES, check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# rows, q heads, k heads, head_dim, rotary_dim
SHAPES = [(1, 32, 8, 128, 128), (1, 1, 1, 2, 2), (7, 4, 2, 80, 32), (33, 3, 1, 96, 50), (5, 2, 2, 10, 6),
          (64, 32, 32, 128, 64), (300, 5, 5, 72, 72), (3, 7, 1, 256, 256), (9, 2, 1, 33, 32),
          (2, 1, 1, 1024, 1024), (2, 1, 2, 1024, 2), (2, 2, 1, 1023, 4), (2100, 4, 1, 64, 64),
          (5000, 2, 1, 128, 96), (3, 40, 0, 128, 128), (3, 0, 2, 64, 32), (1300, 3, 1, 512, 512), (11, 2, 2, 32, 32)]


def _inputs(R, Hq, Hk, D, dt, seed, weights=True):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen).to(DTYPES[dt]).to(DEV)
    qkv = rand(R, Hq + 2 * Hk, D)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]  # views of the fused projection
    wq, wk = ((1 + 0.5 * torch.randn(2, D, generator=gen)).to(DTYPES[dt]).to(DEV)) if weights else (None, None)
    pos = torch.randint(0, 50000, (R,), generator=gen).to(DEV)
    return q, k, wq, wk, pos, rand(R, Hq, D), rand(R, Hk, D)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("R,Hq,Hk,D,rot", SHAPES)
def test_forward_and_gradients(R, Hq, Hk, D, rot, layout, dt):
    q, k, wq, wk, pos, dq, dk = _inputs(R, Hq, Hk, D, dt, R + D)
    plan = sg.rope_plan(rot, layout=layout, scaling={"kind": "by_parts", "factor": 4.0, "context": 4096},
                        device=DEV)
    got = sg.qk_norm_rope(q, k, wq, wk, pos, plan, eps=1e-5)
    leaves = [t.detach().requires_grad_() for t in (q, k, wq, wk)]
    grads = torch.autograd.grad(sg.qk_norm_rope(*leaves, pos, plan, eps=1e-5), leaves, [dq, dk])
    for i, (x, w, d) in enumerate(((q, wq, dq), (k, wk, dk))):
        check(got[i], *norm_forward(x, w, pos, plan, 1e-5), f"out {i}")
        (dx, bx), (dw, bw) = norm_backward(x, w, d, pos, plan, 1e-5)
        check(grads[i], dx, bx, f"dx {i}")
        check(grads[2 + i], dw, bw, f"dw {i}")


def test_without_weights_and_one_side():
    q, k, wq, wk, pos, dq, dk = _inputs(20, 4, 2, 64, "bf16", 1)
    plan = sg.rope_plan(64, device=DEV)
    both = sg.qk_norm_rope(q, k, None, None, pos, plan)
    check(both[0], *norm_forward(q, None, pos, plan, 1e-6), "no weight")
    one, none = sg.qk_norm_rope(q, None, wq, None, pos.int(), plan)
    assert none is None and torch.equal(one, sg.qk_norm_rope(q, k, wq, wk, pos, plan)[0])
    # every subset of what needs a gradient gets the same ones
    args = [t.detach() for t in (q, k, wq, wk)]
    leaves = [t.clone().requires_grad_() for t in args]
    want = torch.autograd.grad(sg.qk_norm_rope(*leaves, pos, plan), leaves, [dq, dk])
    for mask in range(1, 16):
        part = [t.clone().requires_grad_(bool(mask >> i & 1)) for i, t in enumerate(args)]
        out = sg.qk_norm_rope(*part, pos, plan)
        for i in (0, 1):
            assert out[i].requires_grad == bool(mask >> i & 5)
        live = [(o, d) for o, d in zip(out, (dq, dk)) if o.requires_grad]
        need = [t for t in part if t.requires_grad]
        got = torch.autograd.grad([o for o, _ in live], need, [d for _, d in live])
        for g, w in zip(got, [w for i, w in enumerate(want) if mask >> i & 1]):
            assert torch.equal(g, w), mask


def test_differences():
    """The gradient against central differences, in float32 along random directions: a step of
    2^-8 leaves a third derivative's 2^-16 and the outputs' rounding over the step, 2^-24 2^8
    of a loss of about 100 terms."""
    q, k, wq, wk, pos, dq, dk = _inputs(6, 3, 2, 48, "f32", 2)
    plan = sg.rope_plan(32, layout="interleaved", device=DEV)
    args = [t.clone().requires_grad_() for t in (q, k, wq, wk)]
    grads = torch.autograd.grad(sg.qk_norm_rope(*args, pos, plan), args, [dq, dk])
    gen = torch.Generator().manual_seed(3)
    dirs = [torch.randn(t.shape, generator=gen).to(DEV) for t in args]

    def loss(h):
        out = sg.qk_norm_rope(*[(t + h * d).detach() for t, d in zip(args, dirs)], pos, plan)
        return sum(float((o.double() * d.double()).sum()) for o, d in zip(out, (dq, dk)))

    h = 2.0 ** -8
    want = (loss(h) - loss(-h)) / (2 * h)
    got = sum(float((g.double() * d.double()).sum()) for g, d in zip(grads, dirs))
    size = sum(float((g.double() * d.double()).abs().sum()) for g, d in zip(grads, dirs))
    assert abs(got - want) <= size * (2.0 ** -10)


def test_in_place_strides_and_alignment():
    plan = sg.rope_plan(64, device=DEV)
    for dt in DTYPES:
        q, k, wq, wk, pos, _, _ = _inputs(20, 8, 2, 64, dt, 4)
        want = sg.qk_norm_rope(q, k, wq, wk, pos, plan)
        base = torch.cat([q, k, k], 1)  # q, k and v heads
        q2, k2 = base[:, :8], base[:, 8:10]
        keep = base[:, 10:].clone()
        got = sg.qk_norm_rope(q2, k2, wq, wk, pos, plan, out=(q2, k2))
        assert got[0] is q2 and torch.equal(q2, want[0]) and torch.equal(k2, want[1])
        assert torch.equal(base[:, 10:], keep)
    gen = torch.Generator().manual_seed(5)
    w = torch.randn(64, generator=gen).half().to(DEV)
    pos = torch.randint(0, 999, (11,), generator=gen).to(DEV)
    off = torch.randn(11 * 3 * 64 + 3, generator=gen).half().to(DEV)[3:].view(11, 3, 64)
    for x in (torch.randn(5, 11, 64, generator=gen).half().to(DEV).transpose(0, 1), off,
              torch.randn(11, 3, 70, generator=gen).half().to(DEV)[..., 1:65],
              torch.randn(1, 1, 64, generator=gen).half().to(DEV).expand(11, 4, 64)):
        check(sg.qk_norm_rope(x, None, w, None, pos, plan)[0], *norm_forward(x, w, pos, plan, 1e-6), "strides")
    # gradients that repeat or lie otherwise than the inputs
    leaf, wl = off.clone().requires_grad_(), w.clone().requires_grad_()
    out = sg.qk_norm_rope(leaf, None, wl, None, pos, plan)[0]
    gx, gw = torch.autograd.grad(out.sum(), [leaf, wl])
    (dx, bx), (dw, bw) = norm_backward(off, w, torch.ones_like(off), pos, plan, 1e-6)
    check(gx, dx, bx, "gradient of a sum")
    check(gw, dw, bw, "weight's gradient of a sum")
    # broadcast inputs: their gradients add up over what they were broadcast to
    one = torch.randn(1, 1, 64, generator=gen).to(DEV).requires_grad_()
    out = sg.qk_norm_rope(one.expand(11, 4, 64), None, None, None, pos, plan)[0]
    d = torch.randn(11, 4, 64, generator=gen).to(DEV)
    g, = torch.autograd.grad(out, [one], d)
    (dx, bx), _ = norm_backward(one.detach().expand(11, 4, 64), None, d, pos, plan, 1e-6)
    check(g, dx.sum((0, 1), keepdim=True), bx.sum((0, 1), keepdim=True) + 44 * 2.0 ** -24 * dx.abs().sum((0, 1), keepdim=True),
          "broadcast")


def test_zeros_and_non_finite():
    plan = sg.rope_plan(16, device=DEV)
    x = torch.zeros(3, 2, 16, device=DEV)
    x[1, 0, 3], x[2, 1, 5] = float("inf"), float("nan")
    pos = torch.arange(3, device=DEV)
    y = sg.qk_norm_rope(x, None, None, None, pos, plan)[0]
    assert not bool(y[0].any()) and not bool(y[1, 1].any()) and not bool(y[2, 0].any())
    assert bool(torch.isnan(y[2, 1]).any()) and bool(torch.isnan(y[1, 0]).any())
    leaf = x[:1].clone().requires_grad_()
    g, = torch.autograd.grad(sg.qk_norm_rope(leaf, None, None, None, pos[:1], plan)[0].sum(), [leaf])
    assert bool(torch.isfinite(g).all()) and bool(g.any())  # 1 / sqrt(eps) times the turned ones
    e = sg.qk_norm_rope(x[:0], x[:0, :0], None, None, pos[:0], plan)
    assert e[0].shape == (0, 2, 16) and e[1].shape == (0, 0, 16)
    w = torch.ones(16, device=DEV, requires_grad=True)
    g, = torch.autograd.grad(sg.qk_norm_rope(x[:0], None, w, None, pos[:0], plan)[0].sum(), [w])
    assert not bool(g.any())


def test_repeatable_graph_and_stream():
    q, k, wq, wk, pos, dq, dk = _inputs(700, 8, 2, 128, "bf16", 6)
    plan = sg.rope_plan(128, device=DEV)
    step = lambda: sg.qk_norm_rope_backward(dq, dk, q, k, wq, wk, pos, plan)
    first = step()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    # forward and backward captured, replayed over changing positions
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = sg.qk_norm_rope(q, k, wq, wk, pos, plan) + step()
    for n in range(3):
        pos.add_(n + 1)
        graph.replay()
        torch.cuda.synchronize()
        want = sg.qk_norm_rope(q, k, wq, wk, pos, plan) + step()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_captured_training_pass():
    """Forward and backward through autograd in one graph: replays against eager passes, with eager
    work between them.  No eager graph of the captured leaves is alive at the capture."""
    q, k, wq, wk, pos, dq, dk = _inputs(130, 6, 2, 64, "bf16", 7)
    plan = sg.rope_plan(64, device=DEV)
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, wq, wk)]
    eager = [t.detach().clone().requires_grad_() for t in leaves]

    def step(v):
        y = sg.qk_norm_rope(*v, pos, plan)
        return [t.detach() for t in y] + list(torch.autograd.grad(y, v, [dq, dk]))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(leaves)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(leaves)
    for _ in range(3):
        with torch.no_grad():
            for t, e in zip(leaves, eager):
                t.mul_(-0.75)
                e.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step(eager)))


def test_refusals():
    plan = sg.rope_plan(64, device=DEV)
    q = torch.zeros(4, 2, 64, device=DEV)
    w, pos = torch.ones(64, device=DEV), torch.arange(4, device=DEV)
    call = lambda q=q, k=None, wq=w, wk=None, p=pos, plan=plan, **kw: sg.qk_norm_rope(q, k, wq, wk, p, plan, **kw)
    for kind, match, kw in ((TypeError, "plan", dict(plan=1)), (ValueError, "must be given", dict(q=None, wq=None)),
                            (ValueError, "needs its", dict(wk=w)), (ValueError, "exceeds", dict(q=q[..., :32])),
                            (ValueError, "q_weight must be", dict(wq=w[:32].contiguous())),
                            (TypeError, "q_weight must be", dict(wq=w.half())),
                            (ValueError, "dense", dict(q=q.new_zeros(4, 2, 128)[..., ::2])),
                            (ValueError, "positions", dict(p=pos[:3].contiguous())),
                            (TypeError, "int32 or int64", dict(p=pos.float())),
                            (ValueError, "disagree", dict(k=q[:3])), (TypeError, "k must be", dict(k=q.half())),
                            (ValueError, "negative", dict(eps=-1.0)), (ValueError, "negative", dict(eps=float("nan"))),
                            (ValueError, "out q", dict(out=(q[:, :1], None))),
                            (ValueError, "repeat", dict(out=(q[:1].expand(4, 2, 64), None))),
                            (ValueError, "rows, heads", dict(q=q[0])),
                            (ValueError, "recorded", dict(q=q.clone().requires_grad_(), out=(q, None)))):
        with pytest.raises(kind, match=match):
            call(**kw)
    leaf = torch.randn(4, 2, 64, device=DEV).requires_grad_()
    with pytest.raises(RuntimeError, match="once"):
        torch.autograd.grad(sg.qk_norm_rope(leaf, None, w, None, pos, plan)[0].square().sum(), [leaf], create_graph=True)
