"""examples/adapted_layer.py: the operators run together, against the layer's plain 64-bit form."""
import importlib.util
import math
import os

import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from proj_helpers import q4_parts

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapted_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("adapted_layer", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _plain_layer(layer, x, positions, row_ids):
    """The layer in float64 on the CPU."""
    W = {}
    for name, raw in layer.raw.items():
        q, z, s = q4_parts(raw, 2 * raw[0].shape[1], layer.group)
        W[name] = (q - z) * s
    x, ids = x.double().cpu(), row_ids.long().cpu()

    def adapt(x, name):
        A, B = (t.double().cpu()[ids] for t in layer.lora[name])
        return torch.matmul(torch.matmul(x[:, None], A), B)[:, 0]

    def turn(t):
        a = positions.double().cpu()[:, None, None] * layer.plan.inv_freq.double().cpu()
        lo, hi = t.chunk(2, -1)
        m = float(layer.plan.magnitude)
        return m * torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)

    R = x.shape[0]
    heads = lambda t: t.view(R, layer.heads, -1)
    q, k, v = (heads(x @ W[n].t() + (adapt(x, n) if n != "k" else 0)) for n in "qkv")
    q, k, v = (t.transpose(0, 1) for t in (turn(q), turn(k), v))
    s = q @ k.transpose(1, 2) / math.sqrt(q.shape[2])
    s = s.masked_fill(torch.ones(R, R, dtype=torch.bool).triu(1), float("-inf"))
    a = x + (s.softmax(-1) @ v).transpose(0, 1).reshape(R, -1) @ W["o"].t()
    g, u = a @ W["gate"].t() + adapt(a, "gate"), a @ W["up"].t() + adapt(a, "up")
    return a + (g * torch.sigmoid(g) * u) @ W["down"].t()


@pytest.mark.parametrize("R,hidden,ffn", [(1, 128, 344), (33, 256, 688), (90, 128, 200)])
def test_served_layer(example, R, hidden, ffn):
    layer = example.AdaptedLayer(hidden, ffn, heads=4, adapters=5, rank=8, dtype=torch.float32, seed=R)
    gen = torch.Generator().manual_seed(R)
    x = torch.randn(R, hidden, generator=gen).cuda()
    positions = torch.arange(R, device="cuda") + 1000
    row_ids = torch.randint(0, 5, (R,), generator=gen, dtype=torch.int32).sort().values.cuda()
    seg, ids, _ = sg.build_segments(row_ids, 5)
    y = layer.serve(x, positions, (seg, ids))
    ref = _plain_layer(layer, x, positions, row_ids)
    # Eight stages in a row; in each a float32 sum of at most 700 terms is off by
    # 700 2^-24 = 4e-5 of its terms' magnitudes, of which sums of independent terms are a
    # tenth or more, and the softmax and the activation stretch an error by a few times.
    assert float((y.double().cpu() - ref).norm() / ref.norm()) <= 8 * 10 * 4e-5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_training_lowers_the_loss(example, dtype):
    layer = example.AdaptedLayer(256, 520, heads=4, adapters=2, rank=8, dtype=dtype)
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(130, 256, generator=gen).to(dtype).cuda()
    target = torch.randn(130, 520, generator=gen).to(dtype).cuda()
    losses = example.train_block(layer, x, target, adapter=1, steps=10)
    assert all(math.isfinite(v) for v in losses) and losses[-1] < losses[0]


def test_main_runs(example, capsys):
    example.main()
    assert "trained 20 steps" in capsys.readouterr().out
