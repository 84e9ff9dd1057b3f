"""The plan made on the device is cut as the plain model says, whose room the CPU tests check, and its results are
right where some rows are joined and others are not."""
import random

import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from attention_plan_model import cut, draw, reserved, widest
from proj_helpers import DTYPES
from test_gpu_prefix_attention import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dim,dt", [(64, "f16"), (128, "f32"), (256, "bf16")])
def test_items_and_slots(dim, dt):
    rng = random.Random(dim)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    code = {"f32": 0, "f16": 1, "bf16": 2}[dt]
    for _ in range(60):
        rows, tokens, cuts, prefix, rep, heads = draw(rng)
        cache = sg.kv_cache(1, 16, heads, dim, DTYPES[dt], device=DEV)
        if sum(rows) == 0 or reserved(sg.lib(), cache._c, sum(rows), len(rows), len(prefix), rep * heads, code) is None:
            continue
        first = [0]
        for r in rows:
            first.append(first[-1] + r)
        width = lambda lengths: -(-max(lengths) // 16)
        kw = {}
        if prefix:
            kw = dict(prefix_pages=torch.zeros(len(prefix), width(prefix), dtype=torch.int32, device=DEV),
                      prefix_lengths=i32(prefix), prefix_indptr=i32(cuts))
        plan = sg.prefix_plan(cache, rep * heads, torch.zeros(len(rows), width(tokens), dtype=torch.int32, device=DEV),
                              i32(tokens), row_indptr=i32(first), num_rows=sum(rows), **kw)
        got = tuple(plan.table[:8].view(torch.int32).tolist())
        assert got == cut(rows, tokens, cuts, prefix, rep, heads, widest(dim, code)), (rows, tokens, cuts, prefix)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("cuts,prefix", [([], []), ([0, 2], [150])])
def test_joined_and_not(cuts, prefix, dt):
    """One long sequence that is cut among short ones that are not, prompts and single rows."""
    b = Batch([1, 40, 1, 3, 1], [6000, 40, 9, 3, 0], cuts, prefix, 8, 2, 64, 16, "fp8", dt, seed=80)
    b.verify("mixed")
    b = Batch([35, 1], [9000, 20], cuts, prefix, 4, 1, 128, 64, "fp4", dt, seed=81)
    b.verify("a long prompt")
