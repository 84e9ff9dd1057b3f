"""Sizes past 32 bits are refused: cut off, 2^32 + 1 pages would be one."""
import types

import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from segmented_gather_gemv_sgmv_amd import attention, kv, norm

CPU = torch.device("cpu")


def test_caches():
    for name in ("num_pages", "page_size", "kv_heads", "head_dim"):
        for big in (2 ** 31, 2 ** 32 + 16, -(2 ** 32) + 16):
            args = dict(num_pages=16, page_size=16, kv_heads=16, head_dim=16, dtype=torch.float32, device="cpu")
            args[name] = big
            with pytest.raises(ValueError, match=f"{name} must be below"):
                sg.kv_cache(**args)


def _shape(*shape):
    """What the checks look at, without the memory."""
    return types.SimpleNamespace(shape=torch.Size(shape), dtype=torch.int32, device=CPU, dim=lambda: len(shape))


def test_rows(monkeypatch):
    cache, one_head = sg.kv_cache(2, 16, 1, 64, torch.float32, device="cpu"), torch.zeros(1, 1, 2)
    for module in (kv, norm, attention):
        monkeypatch.setattr(module, "_need", lambda *a: None)
    with pytest.raises(ValueError, match="rows must be below"):
        kv._slots(cache, _shape(2 ** 32 + 3))
    assert kv._slots(cache, _shape(2 ** 31 - 1)) == 2 ** 31 - 1
    for shape, name in (((2 ** 32 + 1, 1, 2), "rows"), ((1, 2 ** 32 + 1, 2), "heads"), ((1, 1, 2 ** 32 + 2), "head_dim")):
        with pytest.raises(ValueError, match=f"{name} must be below"):
            norm._common(_shape(*shape), None, None, None, _shape(shape[0]), None)
    many = (None, 0, 0, (0, 0, 0, 0), 2 ** 32 + 1)  # heads of k, which _common does not look at
    monkeypatch.setattr(norm, "_common", lambda *a: (CPU, torch.float32, 1, 2))
    monkeypatch.setattr(norm, "_one", lambda t, name, *a: many if name == "k" else (None, 0, 0, (0, 0, 0, 0), 1))
    with pytest.raises(ValueError, match="heads must be below"):
        norm._run(one_head, one_head, None, None, None, None, 0.0, None)
    monkeypatch.setattr(norm, "_side", lambda x, dy, w, want_x, want_w, name, *a: (
        None, None, (None,) * 5, (0,) * 6, 2 ** 32 + 1 if name == "k" else 1))
    with pytest.raises(ValueError, match="heads must be below"):
        norm.qk_norm_rope_backward(one_head, one_head, one_head, one_head, None, None, None, None)
    one, table = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="num_rows must be below"):
        sg.prefix_plan(cache, 1, table, one, num_rows=2 ** 32 + 1)
    with pytest.raises(ValueError, match="q_heads must be below"):
        sg.prefix_plan(cache, 2 ** 32 + 1, table, one)
    with pytest.raises(ValueError, match="pages_per_sequence must be below"):
        sg.prefix_plan(cache, 1, _shape(1, 2 ** 32 + 1), one)
