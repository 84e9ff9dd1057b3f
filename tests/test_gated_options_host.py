"""gated_ffn_backward's options (CPU): refusals and sizes."""
import segmented_gather_gemv_sgmv_amd as sg
from segmented_gather_gemv_sgmv_amd.gated import FULL_GRADIENTS, ONE_WEIGHT

FAKE = 0x1000
R, H, I = 300, 256, 4096


def _backward(dWg=FAKE, dWu=FAKE, dx=FAKE, x=FAKE, dt=1, ws=None, ws_bytes=0):
    return sg.lib().gated_ffn_backward(dx, dWg, dWu, FAKE, FAKE, FAKE, x, FAKE, FAKE, FAKE, FAKE, R, H, I, 0, dt,
                                       ws, ws_bytes, None)


def test_full_gradients():
    size = lambda dt: sg.lib().gated_ffn_backward_workspace_bytes(R, H, I, dt)
    lo = 2 * R * I * 2
    sums = size(1 | FULL_GRADIENTS) - lo  # of ranges, as without, or none
    assert sums >= 0 and sums % (R * H * 4) == 0 and size(2 | FULL_GRADIENTS) == sums + lo
    big = lambda dt: sg.lib().gated_ffn_backward_workspace_bytes(8192, 8192, I, dt)
    assert big(1) == 0 and big(1 | FULL_GRADIENTS) == 2 * 8192 * I * 2
    assert size(FULL_GRADIENTS) == size(0)  # float32 has nothing to add
    assert size(7 | FULL_GRADIENTS) == 0 and size(1 | ONE_WEIGHT) == size(1)
    assert sg.lib().gated_ffn_backward_workspace_bytes(0, H, I, 1 | FULL_GRADIENTS) == 0
    full = 1 | FULL_GRADIENTS
    assert _backward(dt=full) == 5 and _backward(dt=full, ws=FAKE, ws_bytes=size(full) - 1) == 5
    assert _backward(dt=full, dx=None) == 5  # the second parts alone
    assert _backward(dt=full, dx=None, ws=FAKE, ws_bytes=lo - 1) == 5
    assert _backward(dt=full, ws=FAKE + 4, ws_bytes=1 << 30) == 5
    assert _backward(dt=3 | FULL_GRADIENTS) == 3 and _backward(dt=-1) == 3 and _backward(dt=1 | 0x400) == 3


def test_one_weight():
    assert _backward(dWg=None) == 1 and _backward(dWu=None) == 1
    # past that check: the workspace is what is missing
    assert _backward(dWg=None, dt=1 | ONE_WEIGHT) == 5 and _backward(dWu=None, dt=1 | ONE_WEIGHT) == 5
    assert _backward(dWg=None, x=None, dt=1 | ONE_WEIGHT) == 1
    assert _backward(dWu=None, x=None, dt=1 | ONE_WEIGHT) == 1
