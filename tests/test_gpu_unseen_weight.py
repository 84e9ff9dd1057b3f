"""A visible NaN of V makes its rows NaN however small its weight is and however the keys are cut into
items: also where the weight underflows against another item's."""
import math

import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from test_gpu_prefix_attention import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,own,prefix", [([1, 1], [5000, 4000], [3000]), ([40, 33, 2], [2000, 1500, 90], [900])])
def test_nan_of_no_weight(rows, own, prefix, kind, dt):
    """Scores of thousands: one key has all the weight and every other one underflows.  The rows whose
    largest key lies elsewhere see the NaN all the same."""
    b = Batch(rows, own, [0, len(rows)], prefix, 4, 2, 64, 16, kind, dt, seed=60)
    flat = torch.cat(b.slots)
    b.write(flat, (b.k.float() * 100).to(b.dt), b.v)
    n = b.first[-1]
    clean = sg.prefix_attention(b.q, b.cache, b.plan())
    assert bool(torch.isfinite(clean).all())
    # one in the prefix (all rows see it), one in the second sequence's own tokens, ahead of its rows
    second = prefix[0] + own[0]
    for at, seen in ((0, range(n)), (prefix[0] - 1, range(n)), (second, range(b.first[1], b.first[2])),
                     (second + 1000, range(b.first[1], b.first[2]))):
        v = b.v[at: at + 1].clone()
        v[0, 1, 5] = math.nan
        b.write(flat[at: at + 1], (b.k[at: at + 1].float() * 100).to(b.dt), v)
        lse = torch.empty(b.T, 4, device=DEV)
        o = sg.prefix_attention(b.q, b.cache, b.plan(), lse=lse)
        b.write(flat[at: at + 1], (b.k[at: at + 1].float() * 100).to(b.dt), b.v[at: at + 1])
        hit = torch.zeros(n, 4, dtype=torch.bool)
        hit[list(seen), 2:] = True
        assert torch.equal(torch.isnan(o).all(-1).cpu(), hit), at
        assert torch.equal(o[~hit.to(DEV)], clean[~hit.to(DEV)])
        assert bool(torch.isfinite(lse).all())  # the weights are K's alone
