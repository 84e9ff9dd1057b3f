"""The quantized cache: what is read is exactly what the format keeps of what was written."""
import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from attention_helpers import FORMATS, kept
from proj_helpers import DTYPES

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _same(got, want, what=""):
    got, want = got.double().cpu(), want.double()
    ok = (got == want) | (torch.isnan(got) & torch.isnan(want))
    assert bool(ok.all()), (what, int((~ok).sum()), got[~ok][:4], want[~ok][:4])


def _kv(gen, T, H, D, dt, spread=3.0):
    """Values over many magnitudes, a scale of its own for every token."""
    x = torch.randn(2, T, H, D, generator=gen) * torch.exp2(torch.randn(2, T, H, 1, generator=gen) * spread)
    return tuple(x.to(DTYPES[dt]).to(DEV))


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 1, 16), (1, 8, 128, 16), (5, 3, 20, 16), (70, 2, 64, 48),
                                        (33, 4, 80, 32), (64, 1, 96, 64), (130, 2, 112, 16), (300, 2, 128, 128),
                                        (40, 2, 160, 16), (90, 1, 192, 32), (50, 2, 256, 16), (2500, 8, 40, 64)])
def test_round_trip(T, H, D, page, kind, dt):
    gen = torch.Generator().manual_seed(T + D)
    k, v = _kv(gen, T, H, D, dt)
    pages = T // page + 4
    cache = sg.kv_cache(pages, page, H, D, DTYPES[dt], kind, device=DEV)
    want = [kept(t, kind, dt) for t in (k, v)]
    table = torch.randperm(pages, generator=gen)
    for order in ("prompt", "scattered", "shifted"):
        if order == "scattered":
            slots = torch.randperm(pages * page, generator=gen)[:T]
        else:
            t = torch.arange(T) + (0 if order == "prompt" else page // 2 + 1)
            slots = table[t // page] * page + t % page
        for s in (slots.to(DEV), slots.int().to(DEV)):
            before = [t.clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
            sg.kv_write(cache, k, v, s)
            got = sg.kv_read(cache, s)
            for g, w, n in zip(got, want, "kv"):
                _same(g, w, f"{order} {n}")
            # reading in another order, and slots that are not there
            other = torch.randperm(T, generator=gen)
            mixed = torch.cat([slots[other], torch.tensor([-1, pages * page, -5])]).to(DEV)
            for g, w in zip(sg.kv_read(cache, mixed), want):
                _same(g[:T], w[other])
                assert not bool(g[T:].any())
            # what was not named is as it was
            rest = torch.ones(pages * page, dtype=torch.bool)
            rest[slots] = False
            rest = rest.nonzero()[:, 0].to(DEV)
            now = sg.kv_read(cache, rest)
            cache2 = sg.kv_cache(pages, page, H, D, DTYPES[dt], kind, device=DEV)
            for t, b in zip((cache2.k, cache2.v, cache2.k_scales, cache2.v_scales), before):
                t.copy_(b)
            assert all(torch.equal(a, b) for a, b in zip(now, sg.kv_read(cache2, rest)))


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_every_code_tie_and_limit(kind, dt):
    """All codes, all midpoints between them, the group's largest value at and beside every border
    of its exponent, zeros, the type's largest and smallest values, infinities and NaN."""
    grid, group, limits = FORMATS[kind]
    lo, hi = limits[dt]
    f = torch.finfo(DTYPES[dt])
    mids = [(a + b) / 2 for a, b in zip(grid, grid[1:])]
    rows = []
    for e in sorted({lo, lo + 1, -3, 0, 1, hi - 1, hi}):
        for base in (grid, mids):
            part = torch.zeros(128, dtype=torch.float64)
            vals = torch.tensor(base, dtype=torch.float64)[-127:]
            part[:vals.numel()] = vals
            part[1::2] *= -1
            if group:  # one row of a group, its largest code in each
                for at in range(0, 128, 32):
                    part[at: at + 8] = torch.tensor(base + [0.0] * (8 - len(base)), dtype=torch.float64)
            rows.append(part * 2.0 ** e)
            rows.append(-part * 2.0 ** e)
    for v in (0.0, f.max, -f.max, f.tiny, f.smallest_normal * f.eps, 3 * f.smallest_normal * f.eps,
              float("inf"), float("-inf"), float("nan")):
        row = torch.zeros(128, dtype=torch.float64)
        row[37] = v
        row[5] = 1.0
        rows.append(row.clone())
        row[5] = 0.0
        rows.append(row)
    for x in (grid[-1], grid[-1] * (1 + f.eps), grid[-1] * (1 - f.eps), grid[-1] * 2):
        row = torch.full((128,), x, dtype=torch.float64)
        rows.append(row * 0.25)
    x = torch.stack(rows)[:, None].to(DTYPES[dt]).to(DEV)
    n = x.shape[0]
    cache = sg.kv_cache(n // 16 + 1, 16, 1, 128, DTYPES[dt], kind, device=DEV)
    slots = torch.arange(n, device=DEV)
    sg.kv_write(cache, x, -x, slots)
    k, v = sg.kv_read(cache, slots)
    want = kept(x, kind, dt)
    _same(k, want)
    _same(v, -want)


def test_strides_alignment_outputs_and_padding():
    gen = torch.Generator().manual_seed(9)
    qkv = torch.randn(90, 14, 72, generator=gen).bfloat16().to(DEV)
    k, v = qkv[:, 8:11], qkv[:, 11:]
    cache = sg.kv_cache(8, 32, 3, 72, torch.bfloat16, device=DEV)
    slots = torch.arange(90, device=DEV)
    slots[::7] = -1
    slots[3::7] = 256 + 3  # past the cache
    sg.kv_write(cache, k, v, slots)
    live = (slots >= 0) & (slots < 256)
    keep = kept(k, "fp8", "bf16"), kept(v, "fp8", "bf16")
    big = torch.full((90, 5, 75), 7.0, dtype=torch.bfloat16, device=DEV)
    ok, ov = big[:, 1:4, 2:74], torch.empty_like(k)
    got = sg.kv_read(cache, slots, out=(ok, ov))
    assert got[0] is ok
    for g, w in zip(got, keep):
        _same(g[live], w[live.cpu()])
        assert not bool(g[~live].any())
    big[:, 1:4, 2:74] = 7.0
    assert bool((big == 7.0).all())  # nothing beside the view was written
    # heads apart in memory, and one element off the vectors
    x = torch.randn(3, 90, 72, generator=gen).bfloat16().to(DEV).transpose(0, 1)
    off = torch.randn(90 * 3 * 72 + 1, generator=gen).bfloat16().to(DEV)[1:].view(90, 3, 72)
    slots = torch.arange(90, device=DEV) + 100
    sg.kv_write(cache, x, off, slots)
    a, b = sg.kv_read(cache, slots)
    _same(a, kept(x, "fp8", "bf16"))
    _same(b, kept(off, "fp8", "bf16"))
    sg.kv_write(cache, x[:0], off[:0], slots[:0])
    assert sg.kv_read(cache, slots[:0])[0].shape == (0, 3, 72)


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_far_slots(kind):
    """Offsets past 32 bits: codes of K take more than 4 GiB."""
    page, H, D = 128, 8, 256
    pages = (1 << 32) // (page * H * D * (8 if kind == "fp8" else 4) // 8) + 3
    cache = sg.kv_cache(pages, page, H, D, torch.bfloat16, kind, device=DEV)
    gen = torch.Generator().manual_seed(10)
    k, v = _kv(gen, 200, H, D, "bf16")
    slots = torch.cat([torch.arange(100), pages * page - 100 + torch.arange(100)]).to(DEV)
    sg.kv_write(cache, k, v, slots)
    for g, w in zip(sg.kv_read(cache, slots), (k, v)):
        _same(g, kept(w, kind, "bf16"))
    del cache
    torch.cuda.empty_cache()


def test_graph_and_stream():
    gen = torch.Generator().manual_seed(11)
    k, v = _kv(gen, 40, 2, 64, "f16")
    cache = sg.kv_cache(20, 16, 2, 64, torch.float16, "fp4", device=DEV)
    slots = torch.randperm(320, generator=gen)[:40].to(DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sg.kv_write(cache, k, v, slots)
        out = sg.kv_read(cache, slots)
    for n in range(3):
        slots.copy_(torch.randperm(320, generator=gen)[:40])
        k.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        _same(out[0], kept(k, "fp4", "f16"))
        _same(out[1], kept(v, "fp4", "f16"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sg.kv_write(cache, v, k, slots)
        got = sg.kv_read(cache, slots)
    s.synchronize()
    _same(got[0], kept(v, "fp4", "f16"))


def test_refusals():
    cache = sg.kv_cache(4, 16, 2, 64, torch.float16, device=DEV)
    k, slots = torch.zeros(3, 2, 64, device=DEV).half(), torch.arange(3, device=DEV)
    call = lambda c=cache, k=k, v=k, s=slots: sg.kv_write(c, k, v, s)
    for kind, match, kw in ((TypeError, "KVCache", dict(c=1)), (TypeError, "int32 or int64", dict(s=slots.float())),
                            (ValueError, "slots must", dict(s=slots[None])), (TypeError, "k must be", dict(k=k.float())),
                            (ValueError, "v must be", dict(v=k[:2])), (ValueError, "k must be", dict(k=k[:, :1])),
                            (ValueError, "dense", dict(v=k.new_zeros(3, 2, 128)[..., ::2])),
                            (ValueError, "contiguous", dict(s=torch.arange(6, device=DEV)[::2]))):
        with pytest.raises(kind, match=match):
            call(**kw)
    with pytest.raises(RuntimeError, match="no gradients"):
        call(k=k.clone().requires_grad_())
    with pytest.raises(ValueError, match="out v"):
        sg.kv_read(cache, slots, out=(k, k[:2]))
