"""Which views share elements, against the sets of their elements (CPU)."""
import itertools
import random

import pytest
import torch

from segmented_gather_gemv_sgmv_amd.views import apart as _apart, repeats as _repeats, view


def apart(a, b):
    return _apart(view(a), view(b), a.element_size())


def repeats(t):
    return _repeats(view(t))


def _elements(t):
    """Every element's byte address, as a list."""
    r, h, d = t.shape
    s = t.stride()
    return [t.data_ptr() + t.element_size() * (i * s[0] + j * s[1] + k)
            for i, j, k in itertools.product(range(r), range(h), range(d))]


def _view(buf, rng):
    while True:
        shape = (rng.randint(0, 4), rng.randint(1, 4), rng.randint(1, 6))
        stride = (rng.choice([0, 1, 6, 7, 12, 24, 48]), rng.choice([0, 2, 6, 8, 12, 24, 30]), 1)
        at = rng.randint(0, 40)
        if at + sum((max(n, 1) - 1) * s for n, s in zip(shape, stride)) < buf.numel():
            return buf.as_strided(shape, stride, at)


@pytest.mark.parametrize("seed", range(4))
def test_against_the_elements(seed):
    rng, buf = random.Random(seed), torch.zeros(400, dtype=torch.float16)
    told = {True: 0, False: 0}
    for _ in range(1500):
        a, b = _view(buf, rng), _view(buf, rng)
        ea, eb = _elements(a), _elements(b)
        assert repeats(a) == (len(set(ea)) < len(ea)), (a.shape, a.stride())
        want = not set(ea) & set(eb)
        assert apart(a, b) == want and apart(b, a) == want, (a.shape, a.stride(), b.shape, b.stride())
        told[want] += 1
    assert min(told.values()) > 200


def test_views_of_a_fused_buffer():
    qkv = torch.zeros(5, 12, 64)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    assert apart(q, k) and apart(k, v) and apart(v, q) and not apart(q, q) and not repeats(q)
    assert not apart(q, qkv[:, 7:9]) and not apart(qkv[1:, :8], qkv[:-1, :8])
    turned = torch.zeros(12, 5, 64).transpose(0, 1)  # heads outermost
    assert apart(turned[:, :8], turned[:, 8:]) and not apart(turned[:, :8], turned[:, 7:]) and not repeats(turned)
    assert apart(qkv[..., :32], qkv[..., 32:]) and not apart(qkv[..., :33], qkv[..., 32:])
    assert repeats(qkv[:1].expand(5, 12, 64)) and not repeats(qkv[:1])


def test_on_the_host_alone():
    """Addresses are compared on the CPU whatever torch's default device is: a call may be under capture."""
    made = []

    class Mode(torch.overrides.TorchFunctionMode):
        def __torch_function__(self, func, types, args=(), kwargs=None):
            if func is torch.arange:
                made.append((kwargs or {}).get("device"))
            return func(*args, **(kwargs or {}))

    buf = torch.zeros(100)
    a, b = buf.as_strided((3, 2, 4), (8, 12, 1)), buf.as_strided((3, 2, 4), (9, 12, 1), 4)
    with Mode():
        apart(a, b), repeats(a)
    assert made and set(made) == {"cpu"}
