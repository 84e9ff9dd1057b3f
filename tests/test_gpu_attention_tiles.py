"""prefix_attention where many rows share a tile and prefixes stand in front of their sequences'
tokens, against the plain 64-bit form; the norm, the cache and the attention run together."""
import math

import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from attention_helpers import attend, kept, norm_forward
from proj_helpers import DTYPES, check
from test_gpu_prefix_attention import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# Sequences of which each fills a tile of 128 rows (64: float32, heads past 128) read the prefix in front of
# their own tokens; "mixed" has a run where one does not.
FOLDED = {
    "no_prefix": ([40, 33], [90, 33], [0, 2], [0], 8, 2, 64, 16),
    "prefix_1": ([40, 33], [90, 33], [0, 2], [1], 8, 2, 64, 16),
    "prefix_63": ([40, 33], [64, 100], [0, 2], [63], 8, 2, 64, 16),
    "prefix_64": ([40, 33], [65, 33], [0, 2], [64], 8, 2, 128, 32),
    "prefix_65": ([40, 33], [127, 70], [0, 2], [65], 8, 2, 128, 48),
    "no_own": ([130, 129], [0, 0], [0, 2], [150], 1, 1, 64, 16),
    "short_own": ([150, 130], [20, 0], [0, 2], [70], 2, 2, 96, 16),  # fewer tokens than rows
    "mixed": ([40, 35, 1, 50], [50, 40, 9, 50], [0, 2, 4], [100, 130], 8, 2, 80, 16),
    "two_runs": ([33, 40, 64], [40, 41, 70], [0, 1, 3], [31, 200], 4, 1, 128, 64),
    "d192": ([70, 66], [90, 66], [0, 2], [77], 2, 2, 192, 16),
    "d256": ([70, 66], [90, 66], [0, 2], [130], 2, 2, 256, 16),
    "big_pages": ([130], [300], [0, 1], [200], 2, 1, 64, 4096),
    "gap": ([40, 0, 33], [90, 50, 33], [0, 3], [130], 8, 2, 112, 160),
}


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("name", FOLDED)
def test_prefix_in_front(name, kind, dt):
    b = Batch(*FOLDED[name], kind, dt, seed=20 + len(name), tail=1)
    out = torch.full((b.T, b.Hq, b.D), 5.0, dtype=b.dt, device=DEV)
    plan = b.plan()
    b.verify(name, plan, out=out)
    assert bool((out[b.first[-1]:] == 5.0).all())
    # the same bits into a strided output, which items write themselves
    big = torch.full((b.T, b.Hq + 2, b.D + 3), 5.0, dtype=b.dt, device=DEV)
    view = big[:, 1:-1, 2:-1]
    sg.prefix_attention(b.q, b.cache, plan, out=view)
    assert torch.equal(view, out)
    view.fill_(5.0)
    assert bool((big == 5.0).all())


@pytest.mark.parametrize("D,tokens", [(64, 9000), (256, 30000)])
def test_more_chunks_than_lanes(D, tokens):
    """One row over more chunks of keys than its result has lanes of four elements."""
    b = Batch([1], [tokens], [], [], 1, 1, D, 64, "fp4", "bf16", seed=31)
    b.verify("many chunks")


class Wide(Batch):
    """Tiles of many rows keep V relative to the largest scale that they meet, of keys that a row
    does not see too: a value whose scale lies 2^32 or more below it is lost, at most 2^-31 of
    the largest value (a scale's largest value is above half of the format's largest times the
    scale), and what is kept is off by 2^-25 units that reach 2^7 times the scale: less.  The weights
    sum to 1."""

    def reference(self, q, scale=None, drop=()):
        o, bound, lse, lse_bound = super().reference(q, scale, drop)
        v = self.held(torch.cat(self.slots))[1].abs().amax((0, 2)).repeat_interleave(self.Hq // self.Hk)
        return o, bound + v[None, :, None] * 2.0 ** -31, lse, lse_bound


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_magnitudes_in_wide_tiles(kind, dt):
    big = {"f16": 6, "bf16": 30, "f32": 30}[dt]
    b = Wide([40, 33, 1], [90, 133, 60], [0, 2], [200], 4, 1, 64, 16, kind, dt, seed=32)
    flat = torch.cat(b.slots)
    n = flat.numel()
    for power in (torch.linspace(-big, big, n), torch.linspace(big, -big, n),
                  torch.where(torch.arange(n) % 97 == 0, float(big), -float(big))):
        v = (b.v.float() * torch.exp2(power.round().to(DEV))[:, None, None]).to(b.dt)
        b.write(flat, b.k, v)
        b.verify("magnitudes")
    b.write(flat, b.k, b.v)
    b.verify("scale", scale=6.0)
    b.write(flat, (b.k.float() * 100).to(b.dt), b.v)  # scores of thousands: one key each
    b.verify("large scores")


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_non_finite_in_wide_tiles(kind, which):
    """A NaN or an infinity is seen by the rows that see its token: of a prefix in front all, of own
    tokens the later ones."""
    for value in (math.nan, -math.inf):
        b = Batch([70, 66], [100, 66], [0, 2], [130], 4, 2, 64, 16, kind, "bf16", seed=33)
        clean = sg.prefix_attention(b.q, b.cache, b.plan())
        flat = torch.cat(b.slots)
        for at, rows in ((129, range(136)), (0, range(136)), (130 + 64, range(34, 70)), (229, range(69, 70)),
                         (230 + 5, range(75, 136))):
            k, v = b.k[at: at + 1].clone(), b.v[at: at + 1].clone()
            (k if which == "k" else v)[0, 1, 5] = value
            b.write(flat[at: at + 1], k, v)
            o = sg.prefix_attention(b.q, b.cache, b.plan())
            b.write(flat[at: at + 1], b.k[at: at + 1], b.v[at: at + 1])
            hit = torch.zeros(136, 4, dtype=torch.bool)
            hit[list(rows), 2:] = True
            assert torch.equal(torch.isnan(o).all(-1).cpu(), hit), (value, at)
            assert torch.equal(o[~hit.to(DEV)], clean[~hit.to(DEV)])


def test_pages_outside_the_cache_in_wide_tiles():
    b = Batch([40, 33], [100, 60], [0, 2], [130], 8, 2, 64, 16, "fp8", "f16", seed=34)
    drop = []
    for table, i, j, page in ((b.own_table, 0, 1, -1), (b.own_table, 1, 3, 10 ** 6), (b.prefix_table, 0, 8, 2 ** 30),
                              (b.prefix_table, 0, 2, b.cache.num_pages)):
        s = b.slots[i + 1 if table is b.own_table else 0]
        drop.append(s[16 * j: 16 * (j + 1)])
        table[i, j] = page
    b.verify("bad pages", drop=torch.cat(drop))


def test_lengths_past_the_table_in_wide_tiles():
    b = Batch([130, 130], [160, 144], [0, 2], [64], 2, 2, 64, 16, "fp4", "f16", seed=35, slack=0)
    b.own = [160, 160]
    want = sg.prefix_attention(b.q, b.cache, b.plan())
    b.own, b.prefix = [10 ** 9, 2 ** 31 - 1], [2 ** 31 - 1]
    assert torch.equal(sg.prefix_attention(b.q, b.cache, b.plan()), want)
    b.own, b.prefix = [-3, 160], [-1]
    assert not bool(sg.prefix_attention(b.q, b.cache, b.plan())[:130].any())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("power", [-100.0, 100.0])
def test_very_small_and_large_values(kind, dt, power):
    """Far from 1, yet of one magnitude: rows of wide and of narrow tiles."""
    b = Batch([40, 1, 33, 5], [90, 60, 40, 9], [0, 2, 4], [100, 70], 4, 1, 64, 16, kind, dt, seed=37)
    b.write(torch.cat(b.slots), b.k, (b.v.float() * 2.0 ** power).to(b.dt))
    b.verify("power")


def test_outputs_over_inputs_are_refused():
    b = Batch([1, 1], [5, 9], [], [], 2, 2, 64, 16, "fp8", "f16", seed=36)
    with pytest.raises(ValueError, match="apart"):
        sg.prefix_attention(b.q, b.cache, b.plan(), out=b.q)


def test_outputs_that_repeat_are_refused():
    b = Batch([1, 1], [5, 9], [], [], 2, 2, 64, 16, "fp8", "f16", seed=36)
    same = torch.zeros(1, 2, 64, device=DEV).half().expand(2, 2, 64)
    with pytest.raises(ValueError, match="repeat"):
        sg.prefix_attention(b.q, b.cache, b.plan(), out=same)
    slots = torch.tensor([0, 1], device=DEV)
    with pytest.raises(ValueError, match="repeat"):
        sg.kv_read(b.cache, slots, out=(torch.zeros(2, 2, 64, device=DEV).half(), same))


@pytest.mark.parametrize("kind,dt,Hq,Hk,D,rot", [("fp8", "bf16", 8, 2, 128, 128), ("fp4", "f16", 4, 4, 64, 64),
                                                 ("fp8", "f32", 6, 2, 80, 32), ("fp4", "bf16", 5, 1, 192, 96)])
def test_a_step_together(kind, dt, Hq, Hk, D, rot):
    """Norm and rotation, the rows' keys and values into the cache, attention over it: eager, each
    against its plain form of what it was given, then captured and replayed with new rows, positions, slots and
    lengths, which has to give the eager bits."""
    dtype, S, page, eps = DTYPES[dt], 5, 16, 1e-5
    gen = torch.Generator().manual_seed(40)
    plan = sg.rope_plan(rot, device=DEV)
    weights = [(1 + 0.2 * torch.randn(D, generator=gen)).to(dtype).to(DEV) for _ in range(2)]
    prefix, own = 37, [3, 16, 1, 30, 18]
    cache = sg.kv_cache(3 + 3 * S, page, Hk, D, dtype, kind, device=DEV)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    table = i32([[4, 0, 9]])
    free = [p for p in torch.randperm(3 + 3 * S, generator=gen).tolist() if p not in (4, 0, 9)]
    pages = i32(free).view(S, 3)
    fresh = lambda n, H: torch.randn(n, H, D, generator=gen).to(dtype).to(DEV)
    place = lambda row, t: (row.long()[t // page] * page + t % page)
    before = [place(table[0], torch.arange(prefix, device=DEV))]
    before += [place(pages[s], torch.arange(own[s] - 1, device=DEV)) for s in range(S)]
    for slots in before:
        sg.kv_write(cache, fresh(slots.numel(), Hk), fresh(slots.numel(), Hk), slots)

    qkv = fresh(S, Hq + 2 * Hk)  # a fused projection's output
    lengths, positions = i32(own), i32([prefix + n - 1 for n in own])
    slots = torch.stack([place(pages[s], torch.tensor(own[s] - 1, device=DEV)) for s in range(S)])

    def step():
        q, k = sg.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq: Hq + Hk], *weights, positions, plan, eps=eps)
        sg.kv_write(cache, k, qkv[:, Hq + Hk:], slots)
        p = sg.prefix_plan(cache, Hq, pages, lengths, prefix_pages=table, prefix_lengths=i_prefix)
        return q, k, sg.prefix_attention(q, cache, p)

    i_prefix = i32([prefix])
    q, k, o = step()
    for x, y, w in ((qkv[:, :Hq], q, weights[0]), (qkv[:, Hq: Hq + Hk], k, weights[1])):
        check(y, *norm_forward(x, w, positions, plan, eps), "norm")
    held = sg.kv_read(cache, slots)
    for x, y in zip((k, qkv[:, Hq + Hk:]), held):
        assert torch.equal(y.double().cpu(), kept(x, kind, dt))
    for s in range(S):
        every = torch.cat([before[0], before[1 + s], slots[s: s + 1]])
        kk, vv = (t.double().cpu().repeat_interleave(Hq // Hk, 1) for t in sg.kv_read(cache, every))
        ref, bound, _, _ = attend(q[s: s + 1], kk, vv, 1 / math.sqrt(D))
        check(o[s: s + 1], ref, bound, "attention")

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for n in range(3):
        qkv.copy_(fresh(S, Hq + 2 * Hk))
        lengths.add_(1)
        positions.add_(1)
        slots.copy_(torch.stack([place(pages[s], lengths[s].long() - 1) for s in range(S)]))
        graph.replay()
        torch.cuda.synchronize()
        captured = [t.clone() for t in got] + list(sg.kv_read(cache, slots))
        eager = list(step()) + list(sg.kv_read(cache, slots))
        assert all(torch.equal(x, y) for x, y in zip(captured, eager)), n
