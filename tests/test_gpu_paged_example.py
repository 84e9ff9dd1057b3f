"""examples/adapted_layer.py over a paged cache: the layer's steps against its plain 64-bit form."""
import importlib.util
import math
import os

import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from proj_helpers import q4_parts

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapted_layer.py")
spec = importlib.util.spec_from_file_location("adapted_layer", PATH)
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


class Plain:
    """The layer in float64 on the CPU, a row at a time, over given keys and values."""

    def __init__(self, layer):
        self.layer, self.W = layer, {}
        for name, raw in layer.raw.items():
            q, z, s = q4_parts(raw, 2 * raw[0].shape[1], layer.group)
            self.W[name] = (q - z) * s

    def adapt(self, x, name, i):
        if i < 0:
            return 0.0
        A, B = (t[i].double().cpu() for t in self.layer.lora[name])
        return x @ A @ B

    def heads(self, x, position, i):
        """(q, k, v) [heads, D] of a row x [hidden] with adapter i."""
        L = self.layer
        q, k, v = ((self.W[n] @ x + (self.adapt(x, n, i) if n != "k" else 0)).view(L.heads, -1) for n in "qkv")

        def turn(t, w):
            t = t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w.double().cpu()
            a = position * L.plan.inv_freq.double().cpu()
            lo, hi = t.chunk(2, -1)
            return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1) * float(L.plan.magnitude)

        return turn(q, L.norms["q"]), turn(k, L.norms["k"]), v

    def finish(self, x, q, keys, values, i):
        """The layer's output from q and the keys and values [n, heads, D] that it sees."""
        s = torch.einsum("hd,nhd->hn", q, keys) / math.sqrt(q.shape[1])
        a = x + self.W["o"] @ torch.einsum("hn,nhd->hd", s.softmax(-1), values).flatten()
        g, u = (self.W[n] @ a + self.adapt(a, n, i) for n in ("gate", "up"))
        return a + self.W["down"] @ (g * torch.sigmoid(g) * u)


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_steps_over_the_cache(kind):
    hidden, heads, n, S = 256, 4, 21, 6
    layer = example.AdaptedLayer(hidden, 520, heads=heads, adapters=3, rank=8, dtype=torch.float32, seed=2)
    gen = torch.Generator().manual_seed(2)
    prompt, rows = torch.randn(n, hidden, generator=gen).cuda(), torch.randn(S, hidden, generator=gen).cuda()
    row_ids = torch.tensor([0, 0, 1, 1, 1, 2], dtype=torch.int32, device="cuda")
    seg, ids, _ = sg.build_segments(row_ids, 3)
    seen = []
    serve = layer.serve_cached
    layer.serve_cached = lambda x, *rest: seen.append((x, serve(x, *rest))) or seen[-1][1]
    y, cache, at, slots = example.serve_batch(layer, prompt, rows, 3, (seg, ids), kind)
    assert len(seen) == 4 and torch.equal(y, seen[-1][1])
    plain = Plain(layer)
    held = lambda s: [t.double().cpu() for t in sg.kv_read(cache, s)]

    def compare(x, got, positions, adapters, before):
        ref, keys = [], []
        for r in range(x.shape[0]):
            xr = x[r].double().cpu()
            q, k, v = plain.heads(xr, float(positions[r]), adapters[r])
            ref.append(plain.finish(xr, q, *held(before[r]), adapters[r]))
            keys.append((k, v))
        ref = torch.stack(ref)
        # Six stages of at most 520 terms, 520 2^-24 = 3.1e-5 of their magnitudes each; sums of independent
        # terms are a tenth of these or more, and softmax and activation stretch an error by a few times.
        assert float((got.double().cpu() - ref).norm() / ref.norm()) <= 6 * 10 * 3.1e-5
        return [torch.stack(t) for t in zip(*keys)]

    def in_the_cache(want, slots):
        # half a step of the codes (e4m3 2^-4; e2m1 a quarter of the value, or of the least one, which is a twelfth
        # of the largest at most), and the errors above ahead of them
        for w, got in zip(want, held(slots)):
            step = 2.0 ** -4 if kind == "fp8" else 0.25
            floor = 2.0 ** -17 if kind == "fp8" else 1 / 12
            top = w.abs().amax(-1, keepdim=True)
            assert bool(((got - w).abs() <= step * w.abs() + (floor + 2e-3) * top).all())

    x, got = seen[0]
    in_the_cache(compare(x, got, range(n), [-1] * n, [at[: r + 1] for r in range(n)]), at)
    for t, (x, got) in enumerate(seen[1:]):
        before = [torch.cat([at, slots[s, : t + 1]]) for s in range(S)]
        in_the_cache(compare(x, got, [n + t] * S, row_ids.tolist(), before), slots[:, t].contiguous())


def test_main_decodes(capsys):
    example.main()
    assert "decoded 8 steps of 40 sequences" in capsys.readouterr().out
