"""4-bit projections by strips, over every count of K blocks per wave group:
the loop's steps and each of the steps that follow it, on exact sums."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from exact_helpers import check_exact, check_product, exact_q4, exact_sum, exact_x
from proj_helpers import DTYPES

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _both(R, K, N, G, dt):
    gen = torch.Generator().manual_seed(K + R)
    dtype = DTYPES[dt]
    wg, wu = (exact_q4(gen, N, K, G, dtype, z, DEV) for z in (True, False))
    x = exact_x(gen, R, K, dtype, DEV)
    pg, pu = (sg.q4_pack(*w, group_size=G, in_features=K) for w in (wg, wu))
    g, u = (exact_sum(x, w, K, G) for w in (wg, wu))
    check_exact(sg.q4_linear(x, pg), g, f"q4_linear {R}x{K}->{N} G={G}")
    check_product(sg.q4_gated_ffn(x, pg, pu, "relu"), g, u, f"q4_gated_ffn {R}x{K}->{N} G={G}")


# 40 features take eight wave groups, three blocks of x ahead; a block is 128 of K,
# of each of the groups in turn.
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("K", [1000, 1024, 1032, 2048, 2064, 3072, 3080, 4104, 5120, 5128, 6152, 7000])
def test_few_features(K, G, dt):
    _both(9, K, 40, G, dt)


# 13000 features take one wave group, two blocks ahead; between, two and four groups.
@pytest.mark.parametrize("N", [2900, 5500, 13000])
@pytest.mark.parametrize("R", [9, 30, 70])
@pytest.mark.parametrize("K", [120, 256, 376, 512, 1160])
def test_more_features(K, R, N):
    _both(R, K, N, 128, "bf16")
    _both(R, K, N, 32, "f16")
