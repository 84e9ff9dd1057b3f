"""The weights' gradients over many rows: what workgroups found is added without losing the small ones."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("rows", [70, 500, 1003, 1024])
@pytest.mark.parametrize("first", [0, 5, 69])
def test_one_large_row_among_small_ones(rows, first):
    """x = (1, 1), eps = 0 and position 0: the gradient is the plain sum of dy.  Up to 1024 rows are one a workgroup,
    whose sums are exact here; the sum over them is rounded to float32 once: half a step, 2^-24 of it."""
    x = torch.ones(rows, 1, 2, device=DEV)
    dy = torch.ones(rows, 1, 2, device=DEV)
    dy[:, 0, 1] = -3.0
    dy[first, 0] = torch.tensor([2.0 ** 24, 2.0 ** 30 + 128], device=DEV)
    w = torch.ones(2, device=DEV)
    plan = sg.rope_plan(2, device=DEV)
    pos = torch.zeros(rows, dtype=torch.int64, device=DEV)
    for q, k in ((x, None), (None, x)):
        dw = sg.qk_norm_rope_backward(*(None if t is None else dy for t in (q, k)), q, k, None if q is None else w,
                                      None if k is None else w, pos, plan, eps=0.0,
                                      need=(False, False, True, True))[2 if q is not None else 3].double().cpu()
        want = dy.double().sum((0, 1)).cpu()
        assert bool(((dw - want).abs() <= want.abs() * 2.0 ** -24).all()), (dw - want)
