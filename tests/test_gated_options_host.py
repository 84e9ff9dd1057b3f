"""gated_ffn_backward's options (CPU): refusals and sizes."""
import segmented_gather_gemv_sgmv_amd as sg
from segmented_gather_gemv_sgmv_amd.gated import ONE_WEIGHT

FAKE = 0x1000
R, H, I = 300, 256, 4096


def _backward(dWg=FAKE, dWu=FAKE, dx=FAKE, x=FAKE, dt=1, ws=None, ws_bytes=0):
    return sg.lib().gated_ffn_backward(dx, dWg, dWu, FAKE, FAKE, FAKE, x, FAKE, FAKE, FAKE, FAKE, R, H, I, 0, dt,
                                       ws, ws_bytes, None)


def test_one_weight():
    assert _backward(dWg=None) == 1 and _backward(dWu=None) == 1
    # past that check: the workspace is what is missing
    assert _backward(dWg=None, dt=1 | ONE_WEIGHT) == 5 and _backward(dWu=None, dt=1 | ONE_WEIGHT) == 5
    assert _backward(dWg=None, x=None, dt=1 | ONE_WEIGHT) == 1
    assert _backward(dWu=None, x=None, dt=1 | ONE_WEIGHT) == 1
