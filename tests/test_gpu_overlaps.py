"""Outputs that share elements with what a call still reads, or with each other, are refused; views that
lie between each other in one buffer are not."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from test_gpu_prefix_attention import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_attention_into_its_queries():
    b = Batch([3, 2], [20, 9], [0, 2], [70], 4, 2, 64, 16, "fp8", "f16", seed=70)
    plan, T = b.plan(), b.T
    want = sg.prefix_attention(b.q, b.cache, plan)
    big = torch.zeros(T + 1, 9, 64, dtype=torch.float16, device=DEV)
    q = big[:T, :4]
    q.copy_(b.q)
    before = big.clone()
    for out in (q, big[1:, :4], big[:T, 1:5], big[:T, 3:7], big[1:, 2:6], big.flatten()[8:8 + T * 256].view(T, 4, 64)):
        with pytest.raises(ValueError, match="apart"):
            sg.prefix_attention(q, b.cache, plan, out=out)
    assert torch.equal(big, before)  # refused ahead of any work
    for out in (big[:T, 4:8], big[1:, 5:]):
        assert torch.equal(sg.prefix_attention(q, b.cache, plan, out=out), want)
        assert torch.equal(q, b.q)


def test_outputs_of_a_read():
    b = Batch([1, 1], [20, 9], [], [], 2, 2, 64, 16, "fp4", "bf16", seed=71)
    slots = torch.cat(b.slots).to(DEV)
    n = slots.numel()
    want = sg.kv_read(b.cache, slots)
    big = torch.zeros(n + 1, 5, 64, dtype=torch.bfloat16, device=DEV)
    before = big.clone()
    for out in ((big[:n, :2], big[:n, :2]), (big[:n, :2], big[:n, 1:3]), (big[:n, :2], big[1:, :2])):
        with pytest.raises(ValueError, match="apart"):
            sg.kv_read(b.cache, slots, out=out)
    lying = big.flatten().as_strided((n, 2, 64), (96, 64, 1))  # rows run into each other
    for out in ((lying, want[1]), (want[0], lying)):
        with pytest.raises(ValueError, match="repeat"):
            sg.kv_read(b.cache, slots, out=out)
    assert torch.equal(big, before)
    k, v = sg.kv_read(b.cache, slots, out=(big[:n, :2], big[:n, 2:4]))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    with pytest.raises(ValueError, match="out k must be"):
        sg.kv_read(b.cache, slots, out=(big[:1, :2], big[:n, 2:4]))


def test_norm_into_its_inputs():
    """In place, into places of their own in the inputs' buffer, or refused."""
    gen = torch.Generator().manual_seed(72)
    R, D = 9, 64
    data = torch.randn(R + 1, 12, D, generator=gen).half().to(DEV)
    w = torch.ones(D, dtype=torch.float16, device=DEV)
    pos, plan = torch.arange(R, device=DEV), sg.rope_plan(D, device=DEV)
    call = lambda q, k, out: sg.qk_norm_rope(q, k, w, w, pos, plan, out=out)
    want = call(data[:R, :4], data[:R, 4:6], None)

    big = data.clone()
    q, k = big[:R, :4], big[:R, 4:6]
    for out, match in (((q, q[:, :2]), "apart"), ((k.repeat(1, 2, 1), q[:, :2]), "apart"), ((big[1:, :4], k), "apart"),
                       ((big[:R, 1:5], None), "apart"), ((None, big[:R, 5:7]), "apart"), ((big[:R, 6:10], big[:R, 9:11]), "apart"),
                       ((big[:R, 2:6], k), "apart"), ((q, big[1:, 4:6]), "apart"),
                       ((big.flatten().as_strided((R, 4, D), (D, D, 1), 8 * D), k), "repeat"),
                       ((q, big[:1, 8:10].expand(R, 2, D)), "repeat")):
        with pytest.raises(ValueError, match=match):
            call(q, k, out)
    with pytest.raises(ValueError, match="apart"):
        call(q, q, (q, q))  # in place, twice
    assert torch.equal(big, data)

    for out in (lambda b: (b[:R, 6:10], b[:R, 10:12]), lambda b: (b[:R, :4], b[:R, 4:6]), lambda b: (b[:R, :4], None),
                lambda b: (b[:R, 6:10], b[:R, 4:6]), lambda b: (None, b[1:, 7:9])):
        big = data.clone()
        a, b = call(big[:R, :4], big[:R, 4:6], out(big))
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    big = data.clone()
    a, _ = sg.qk_norm_rope(big[:R, :4], None, w, None, pos, plan, out=(big[:R, :4], None))
    assert torch.equal(a, want[0]) and torch.equal(big[:R, 4:], data[:R, 4:])
