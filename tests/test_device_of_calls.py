"""Calls on tensors of another device than the current one launch with theirs as the current one."""
import contextlib

import torch

import segmented_gather_gemv_sgmv_amd as sg


def test_device_is_switched_for_the_call(monkeypatch):
    now = [1]

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], d.index
        yield
        now[0] = before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    seen = []
    for d in (torch.device("cuda", 0), torch.device("cuda", 1), torch.device("cuda")):
        assert sg._call_on(d, lambda x: seen.append(now[0]) or x, 7) == 7
        assert now[0] == 1
    assert seen == [0, 1, 1]
