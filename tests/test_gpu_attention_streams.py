"""Cache, plan and attention on a stream of their own: the bits of the default stream."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from test_gpu_prefix_attention import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("rows,own", [([1, 1, 3], [300, 40, 90]), ([40, 33, 64], [50, 33, 200])])
@pytest.mark.parametrize("kind,dt", [("fp8", "bf16"), ("fp4", "f32")])
def test_another_stream(rows, own, kind, dt):
    b = Batch(rows, own, [0, 3], [150], 4, 2, 64, 16, kind, dt, seed=95)
    lse = torch.empty(b.T, 4, device=DEV)
    want = b.verify("default stream"), sg.kv_read(b.cache, torch.cat(b.slots).to(DEV))
    flat, stream = torch.cat(b.slots).to(DEV), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        b.write(flat, b.k, b.v)
        o = sg.prefix_attention(b.q, b.cache, b.plan(), lse=lse)
        held = sg.kv_read(b.cache, flat)
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(o, want[0]) and all(torch.equal(x, y) for x, y in zip(held, want[1]))
