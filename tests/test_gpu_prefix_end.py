"""Sequences with fewer own tokens than rows, behind a prefix: every row sees all of the prefix, also
those whose place lies before the first own token, however many they are and whether the prefix is read in
front of the sequence's own tokens or apart from them."""
import math

import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from attention_helpers import attend
from proj_helpers import check
from test_gpu_prefix_attention import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Grouped(Batch):
    """Rows that see the same keys are taken together in the reference (Batch's takes one at a time)."""

    def reference(self, q, scale=None, drop=()):
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        outs = []
        for i, n in enumerate(self.rows):
            runs = [g for g in range(len(self.prefix)) if self.cuts[g] <= i < self.cuts[g + 1]]
            slots = self.slots[len(self.prefix) + i]
            before = self.slots[runs[0]] if runs else slots[:0]
            seen = [max(self.own[i] - n + r + 1, 0) for r in range(n)]
            r = 0
            while r < n:
                end = r + seen[r:].count(seen[r])  # they do not decrease
                keys = torch.cat([before, slots[: seen[r]]])
                k, v = (t.repeat_interleave(self.Hq // self.Hk, 1) for t in self.held(keys))
                outs.append(attend(q[self.first[i] + r: self.first[i] + end], k, v, scale))
                r = end
        return [torch.cat(t) for t in zip(*outs)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("rep", [1, 2, 4])
@pytest.mark.parametrize("rows", [160, 300])
def test_all_of_the_prefix(rows, rep, kind, dt):
    for own in (0, 20):
        for prefix in (50, 150):
            b = Grouped([rows], [own], [0, 1], [prefix], rep, 1, 64, 16, kind, dt, seed=50 + own)
            b.verify(f"{own} tokens behind {prefix}")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,rows,own", [(64, 200, 0), (64, 600, 20), (192, 200, 0), (192, 400, 20), (128, 600, 0),
                                        (80, 400, 3), (256, 140, 1)])
def test_heads_and_lengths(D, rows, own, dt):
    b = Grouped([rows, rows + 7], [own, rows], [0, 2], [200], 2, 2, D, 32, "fp8", dt, seed=51, tail=1)
    b.verify("two sequences")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_neighbours_change_nothing(kind, dt):
    """The same sequence in a run of its own and with a short neighbour, which has the prefix
    read apart: both within the bounds, so within both of each other."""
    b = Grouped([160, 1], [20, 9], [0, 2], [150], 4, 1, 64, 16, kind, dt, seed=52)
    together = b.verify("with a short neighbour")
    dev = lambda a: torch.as_tensor(a, dtype=torch.int32).to(DEV)
    plan = sg.prefix_plan(b.cache, 4, dev(b.own_table[:1]), dev([20]), dev([0, 160]), 160, dev(b.prefix_table), dev([150]))
    lse = torch.empty(160, 4, device=DEV)
    alone = sg.prefix_attention(b.q[:160], b.cache, plan, lse=lse)
    ref, bound, ref_lse, lse_bound = (t[:160] for t in b.reference(b.q))
    check(alone, ref, bound, "alone: o")
    check(lse, ref_lse, lse_bound, "alone: lse")
    check(together[:160].double().cpu(), alone.double().cpu(), 2 * bound, "together and alone")
