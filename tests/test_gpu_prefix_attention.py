"""prefix_attention against the plain 64-bit form, over what the cache holds."""
import math

import pytest
import torch

import segmented_gather_gemv_sgmv_amd as sg
from attention_helpers import attend
from proj_helpers import DTYPES, check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Batch:
    """Sequences with rows[i] rows and own[i] tokens, runs of them (cuts) behind prefixes; pages
    anywhere, every slot that holds no token holds NaN."""

    def __init__(self, rows, own, cuts, prefix, Hq, Hk, D, page, kind, dt, seed, tail=0, spread=1.0, slack=2):
        gen = torch.Generator().manual_seed(seed)
        self.rows, self.own, self.cuts, self.prefix = rows, own, cuts, prefix
        self.Hq, self.Hk, self.D, self.dt = Hq, Hk, D, DTYPES[dt]
        counts = prefix + own
        need = [-(-n // page) for n in counts]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=gen)
        self.cache = sg.kv_cache(pages, page, Hk, D, self.dt, kind, device=DEV)
        every = torch.arange(pages * page, device=DEV)
        nan = torch.full((1, Hk, D), math.nan, dtype=self.dt, device=DEV).expand(every.numel(), Hk, D)
        sg.kv_write(self.cache, nan, nan, every)
        width = lambda part: max(part + [0]) + slack
        G = len(prefix)
        self.prefix_table = torch.full((G, width(need[:G])), 10 ** 9)  # past the last token: no page
        self.own_table = torch.full((len(own), width(need[G:])), -7)
        self.slots, at = [], 0
        for i, n in enumerate(counts):
            mine = order[at: at + need[i]]
            at += need[i]
            (self.prefix_table if i < G else self.own_table)[i if i < G else i - G, : need[i]] = mine
            t = torch.arange(n)
            self.slots.append(mine[t // page] * page + t % page)
        n = sum(counts)
        k = torch.randn(n, Hk, D, generator=gen)
        v = torch.randn(n, Hk, D, generator=gen) * torch.exp2(torch.randn(n, Hk, 1, generator=gen) * spread)
        self.k, self.v = k.to(self.dt).to(DEV), v.to(self.dt).to(DEV)
        if n:
            self.write(torch.cat(self.slots), self.k, self.v)
        self.T = sum(rows) + tail
        self.first = [0]
        for r in rows:
            self.first.append(self.first[-1] + r)
        self.q = (torch.randn(self.T, Hq, D, generator=gen) * 1.5).to(self.dt).to(DEV)

    def write(self, slots, k, v):
        sg.kv_write(self.cache, k, v, slots.to(DEV))

    def plan(self, one_row=False):
        dev = lambda a: torch.as_tensor(a, dtype=torch.int32).to(DEV)
        kw = {}
        if self.prefix:
            kw = dict(prefix_pages=dev(self.prefix_table), prefix_lengths=dev(self.prefix),
                      prefix_indptr=dev(self.cuts))
        self.lengths = dev(self.own)
        self.indptr = None if one_row else dev(self.first)
        return sg.prefix_plan(self.cache, self.Hq, dev(self.own_table), self.lengths, row_indptr=self.indptr,
                              num_rows=self.T, **kw)

    def held(self, slots):
        return [t.double().cpu() for t in sg.kv_read(self.cache, slots.to(DEV))]

    def reference(self, q, scale=None, drop=()):
        """(o, bound, lse, bound, covered rows)."""
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        rep = self.Hq // self.Hk
        outs = []
        for i, n in enumerate(self.rows):
            runs = [g for g in range(len(self.prefix)) if self.cuts[g] <= i < self.cuts[g + 1]]
            slots = self.slots[len(self.prefix) + i]
            before = self.slots[runs[0]] if runs else slots[:0]
            for r in range(n):
                seen = torch.cat([before, slots[: max(self.own[i] - n + r + 1, 0)]])
                if len(drop):
                    seen = seen[~torch.isin(seen, drop)]
                k, v = (t.repeat_interleave(rep, 1) for t in self.held(seen))
                row = self.first[i] + r
                outs.append(attend(q[row: row + 1], k, v, scale))
        return [torch.cat(t) for t in zip(*outs)]

    def verify(self, what, plan=None, q=None, scale=None, drop=(), **kw):
        plan = plan or self.plan()
        q = self.q if q is None else q
        lse = torch.full((self.T, self.Hq), 77.0, device=DEV)
        o = sg.prefix_attention(q, self.cache, plan, scale=scale, lse=lse, **kw)
        ref, bound, ref_lse, lse_bound = self.reference(q, scale, drop)
        n = self.first[-1]
        check(o[:n], ref, bound, f"{what}: o")
        empty = torch.isinf(ref_lse)
        assert torch.equal(torch.isinf(lse[:n]).cpu(), empty), what
        check(lse[:n].cpu()[~empty], ref_lse[~empty], lse_bound[~empty], f"{what}: lse")
        assert bool((lse[n:] == 77.0).all())
        return o


# rows, own tokens, first sequences of the runs and the end, prefixes, q heads, k heads, head_dim, page
CASES = {
    "one": ([1], [1], [0, 1], [0], 1, 1, 1, 16),
    "one_long": ([1], [700], [], [], 4, 1, 64, 16),
    "edges": ([1] * 9, [1, 2, 15, 16, 17, 63, 64, 65, 129], [0, 9], [64], 4, 2, 64, 16),
    "prefix_only": ([1, 1, 1], [0, 0, 0], [0, 3], [333], 8, 2, 128, 32),
    "nothing": ([1, 2, 1], [0, 0, 5], [0, 1], [0], 2, 1, 96, 16),
    "chunks": ([5, 1, 0, 17, 40], [5, 90, 30, 17, 130], [0, 5], [200], 6, 2, 80, 48),
    "short_own": ([4, 3], [2, 0], [0, 1], [50], 4, 4, 64, 16),  # fewer tokens than rows
    "runs": ([1, 2, 3, 1, 1, 4], [7, 20, 3, 64, 1, 100], [0, 2, 2, 5], [100, 30, 65], 4, 4, 72, 16),
    "outside": ([1, 1, 1, 1], [10, 20, 30, 40], [1, 3], [90], 8, 8, 40, 16),
    "wide_heads": ([2, 1], [33, 70], [0, 2], [140], 56, 8, 128, 64),
    "d192": ([3, 20], [40, 77], [0, 2], [90], 6, 2, 192, 16),
    "d160": ([1, 1], [100, 300], [0, 2], [64], 5, 1, 160, 128),
    "d256": ([1, 70], [100, 170], [0, 2], [129], 4, 2, 256, 32),
    "d112": ([33, 8], [33, 100], [0, 2], [1], 8, 4, 112, 16),
    "tile_16": ([1] * 16, list(range(16)), [0, 16], [80], 1, 1, 64, 16),
    "tile_17": ([1] * 17, list(range(17)), [0, 17], [80], 1, 1, 64, 16),
    "tile_65": ([13] * 5, [13, 14, 200, 31, 50], [0, 5], [150], 2, 2, 128, 16),
    "tile_129": ([43] * 3, [43, 90, 64], [0, 3], [257], 3, 1, 128, 16),
    "tiles": ([150, 3], [150, 260], [0, 2], [300], 4, 2, 64, 32),
}


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["fp8", "fp4"])
@pytest.mark.parametrize("name", CASES)
def test_against_the_formula(name, kind, dt):
    b = Batch(*CASES[name], kind, dt, seed=len(name), tail=2)
    out = torch.full((b.T, b.Hq, b.D), 5.0, dtype=b.dt, device=DEV)
    plan = b.plan()
    b.verify(name, plan, out=out)
    assert bool((out[b.first[-1]:] == 5.0).all())  # rows of no sequence
    if all(r == 1 for r in b.rows):
        again = b.verify(name + ", a row each", b.plan(one_row=True))
        assert torch.equal(again[: b.first[-1]], out[: b.first[-1]]) and not bool(again[b.first[-1]:].any())
    # the same bits again, and on another stream
    assert torch.equal(sg.prefix_attention(b.q, b.cache, plan)[: b.first[-1]], out[: b.first[-1]])


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_counts_every_key_once(kind):
    """q = 0 weighs all visible keys alike: v that is 1 at one key and 0 elsewhere gives 1 / n there
    and nothing to the rows that do not see it."""
    rows, own, cuts, prefix = [3, 1, 30], [70, 150, 90], [0, 3], [200]
    b = Batch(rows, own, cuts, prefix, 2, 1, 64, 16, kind, "f32", seed=4)
    plan = b.plan()
    q = torch.zeros_like(b.q)
    flat = torch.cat(b.slots)
    zero = torch.zeros(1, 1, 64, device=DEV)
    b.write(flat, zero.expand(flat.numel(), 1, 64), zero.expand(flat.numel(), 1, 64))
    at = [0, 200, 270, 420, 510]  # prefix, then every sequence's tokens
    for key in (0, 15, 16, 63, 64, 199, 200, 263, 264, 267, 268, 269, 270, 400, 419, 420, 479, 480, 481, 509):
        b.write(flat[key: key + 1], zero, zero + 1)
        o = sg.prefix_attention(q, b.cache, plan)
        b.write(flat[key: key + 1], zero, zero)
        for i in range(3):
            for r in range(rows[i]):
                seen = own[i] - rows[i] + r + 1
                mine = key < 200 or at[i + 1] <= key < at[i + 1] + seen
                want = 1 / (200 + seen) if mine else 0.0
                got = o[b.first[i] + r]
                assert bool((got - want).abs().max() <= want * 2.0 ** -20), (key, i, r)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_magnitudes(dt):
    """Values whose scales grow and shrink by 2^20 along the sequence, scores far from 0, scales."""
    big = {"f16": 6, "bf16": 20, "f32": 20}[dt]
    for kind in ("fp8", "fp4"):
        b = Batch([1, 3], [300, 500], [0, 2], [400], 4, 2, 64, 16, kind, dt, seed=5)
        flat = torch.cat(b.slots)
        n = flat.numel()
        for power in (torch.linspace(-big, big, n), torch.linspace(big, -big, n),
                      torch.where(torch.arange(n) % 97 == 0, float(big), -float(big))):
            v = (b.v.float() * torch.exp2(power.round().to(DEV))[:, None, None]).to(b.dt)
            b.write(flat, b.k, v)
            b.verify("magnitudes")
        b.write(flat, b.k, b.v)
        for scale in (1e-4, 1.0, 8.0):
            b.verify("scale", scale=scale)
        b.write(flat, (b.k.float() * 100).to(b.dt), b.v)  # scores of thousands: one key each
        b.verify("large scores")


def test_non_finite():
    """A NaN or an infinity is seen by the rows that see its token, and by no others."""
    for kind in ("fp8", "fp4"):
        for which in ("k", "v"):
            for value in (math.nan, math.inf):
                b = Batch([6, 2], [80, 40], [0, 2], [100], 2, 2, 64, 16, kind, "bf16", seed=6)
                bad = b.slots[1][77:78]  # the row 3 of the first sequence, and later ones, see it
                k, v = b.k[177:178].clone(), b.v[177:178].clone()
                (k if which == "k" else v)[0, 1, 5] = value
                clean = sg.prefix_attention(b.q, b.cache, b.plan())
                b.write(bad, k, v)
                lse = torch.empty(8, 2, device=DEV)
                o = sg.prefix_attention(b.q, b.cache, b.plan(), lse=lse)
                hit = torch.zeros(8, 2, dtype=torch.bool)
                hit[3:6, 1] = True
                assert torch.equal(~torch.isfinite(o).all(-1).cpu(), hit), (kind, which, value)
                assert torch.equal(o[~hit.to(DEV)], clean[~hit.to(DEV)])
                if which == "k":
                    assert torch.equal(torch.isnan(lse).cpu(), hit)


def test_pages_outside_the_cache():
    b = Batch([2, 1], [100, 60], [0, 2], [130], 4, 2, 64, 16, "fp8", "f16", seed=7)
    drop = []
    for table, i, j, page in ((b.own_table, 0, 1, -1), (b.own_table, 1, 3, 10 ** 6), (b.prefix_table, 0, 8, 2 ** 30),
                              (b.prefix_table, 0, 2, b.cache.num_pages)):
        s = b.slots[i + 1 if table is b.own_table else 0]
        drop.append(s[16 * j: 16 * (j + 1)])
        table[i, j] = page
    b.verify("bad pages", drop=torch.cat(drop))


def test_lengths_past_the_table():
    """Lengths are held to what the page tables have room for."""
    b = Batch([1, 1], [48, 32], [0, 2], [64], 2, 2, 64, 16, "fp8", "f16", seed=8, slack=0)
    want = sg.prefix_attention(b.q, b.cache, b.plan())
    b.own, b.prefix = [10 ** 9, 32], [2 ** 31 - 1]
    assert torch.equal(sg.prefix_attention(b.q, b.cache, b.plan()), want)
    b.own, b.prefix = [48, -5], [-1]
    o = sg.prefix_attention(b.q, b.cache, b.plan())
    assert not bool(o[1].any()) and bool(torch.isfinite(o).all())


def test_malformed_rows_stay_inside():
    """Bounds that decrease, overlap or leave the arrays: something finite or nothing at all."""
    b = Batch([4, 4, 4], [30, 40, 50], [0, 3], [70], 4, 2, 64, 16, "fp8", "f16", seed=9)
    for first in ([0, 12, 0, 12], [12, 8, 4, 0], [-5, 4, 400, 12], [0, 10 ** 9, 5, 12]):
        b.first = first
        o = sg.prefix_attention(b.q, b.cache, b.plan(), out=torch.zeros_like(b.q))
        assert bool(torch.isfinite(o).all())
    b.first = [0, 4, 8, 12]
    for cuts in ([3, 0], [-4, 90], [2, 2]):
        b.cuts = cuts
        assert bool(torch.isfinite(sg.prefix_attention(b.q, b.cache, b.plan())).all())


def test_strides_and_alignment():
    for dt in ("bf16", "f32"):
        b = Batch([1, 5, 1], [20, 60, 90], [0, 3], [80], 4, 2, 80, 16, "fp8", dt, seed=10)
        plan = b.plan()
        want = sg.prefix_attention(b.q, b.cache, plan)
        qkv = torch.cat([b.q, torch.zeros(7, 4, 80, dtype=b.dt, device=DEV)], 1)
        off = torch.empty(7 * 4 * 80 + 1, dtype=b.dt, device=DEV)[1:].view(7, 4, 80).copy_(b.q)
        heads = b.q.transpose(0, 1).contiguous().transpose(0, 1)
        for q in (qkv[:, :4], off, heads):
            big = torch.full((7, 6, 83), 3.0, dtype=b.dt, device=DEV)
            out = big[:, 1:5, 2:82]
            assert sg.prefix_attention(q, b.cache, plan, out=out) is out
            assert torch.equal(out, want)
            out.fill_(3.0)
            assert bool((big == 3.0).all())


def test_many_sequences():
    """More sequences than the plan's workgroup has threads, several rounds of items."""
    gen = torch.Generator().manual_seed(11)
    own = torch.randint(0, 40, (2300,), generator=gen).tolist()
    b = Batch([1] * 2300, own, [0, 1000, 1500, 2300], [50, 0, 20], 2, 1, 64, 16, "fp8", "bf16", seed=11)
    b.verify("many sequences")


def test_long_context():
    """Chunks over one long sequence, and a prompt's tiles behind a long prefix."""
    b = Batch([1], [30000], [0, 1], [20000], 2, 2, 128, 64, "fp8", "f16", seed=12)
    b.verify("long decode")
    b = Batch([40], [40], [0, 1], [9000], 8, 1, 128, 64, "fp4", "bf16", seed=13)
    b.verify("long prefix")


def test_far_pages():
    """Offsets past 32 bits: codes of K take more than 4 GiB."""
    page, Hk, D = 128, 8, 256
    pages = (1 << 32) // (page * Hk * D) + 3
    cache = sg.kv_cache(pages, page, Hk, D, torch.float16, device=DEV)
    gen = torch.Generator().manual_seed(14)
    k, v = (torch.randn(150, Hk, D, generator=gen).half().to(DEV) for _ in range(2))
    t = torch.arange(150, device=DEV)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
    slots = table[0].long()[t // page] * page + t % page
    sg.kv_write(cache, k, v, slots)
    q = torch.randn(1, Hk, D, generator=gen).half().to(DEV)
    plan = sg.prefix_plan(cache, Hk, table, torch.tensor([150], dtype=torch.int32, device=DEV))
    o = sg.prefix_attention(q, cache, plan)
    kk, vv = (x.double().cpu() for x in sg.kv_read(cache, slots))
    ref, bound, _, _ = attend(q, kk, vv, 1 / 16)
    check(o, ref, bound, "far pages")
    del cache
    torch.cuda.empty_cache()


def test_graph_with_growing_lengths():
    """Plan and attention captured; replays see new lengths, pages and queries.  Two captured
    graphs and an eager call in between do not disturb one another."""
    b = Batch([1, 1, 1], [30, 100, 64], [0, 3], [90], 4, 2, 64, 16, "fp8", "bf16", seed=15, slack=4)
    dev = lambda a: torch.as_tensor(a, dtype=torch.int32).to(DEV)
    lengths, pages, prefix = dev(b.own), dev(b.own_table), dev(b.prefix_table)
    make = lambda: sg.prefix_plan(b.cache, 4, pages, lengths, prefix_pages=prefix, prefix_lengths=dev_prefix)
    dev_prefix = dev(b.prefix)
    q = b.q.clone()
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plan = make()
            out = sg.prefix_attention(q, b.cache, plan)
        graphs.append((g, out, plan))
    for n in range(3):
        lengths.copy_(dev([30 - 3 * n, 100 - n, 64 - 20 * n]))
        q.add_(0.25)
        for g, _, _ in graphs:
            g.replay()
        eager = sg.prefix_attention(q, b.cache, make())
        torch.cuda.synchronize()
        for _, out, _ in graphs:
            assert torch.equal(out, eager)
        b.own = lengths.tolist()
        b.slots = [b.slots[0]] + [s[:k] for s, k in zip(b.slots[1:], b.own)]
        ref, bound, _, _ = b.reference(q)
        check(eager, ref, bound, f"replay {n}")


def test_two_streams_share_a_plan():
    b = Batch([1, 9, 1], [300, 100, 640], [0, 3], [900], 4, 2, 128, 16, "fp8", "bf16", seed=16)
    plan = b.plan()
    qs = [b.q, b.q * 0.5]
    want = [sg.prefix_attention(q, b.cache, plan) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(sg.prefix_attention(qs[i], b.cache, plan))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)


def test_refusals():
    cache = sg.kv_cache(4, 16, 2, 64, torch.float16, device=DEV)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    pages, lengths = i32([0, 1], [2, 3]), i32(5, 20)
    plan = lambda c=cache, h=4, p=pages, n=lengths, **kw: sg.prefix_plan(c, h, p, n, **kw)
    for kind, match, args in (
            (TypeError, "KVCache", dict(c=1)), (ValueError, "multiple", dict(h=3)), (ValueError, "multiple", dict(h=0)),
            (TypeError, "lengths", dict(n=lengths.long())), (ValueError, "pages must", dict(p=pages[:1])),
            (ValueError, "contiguous", dict(p=pages.t())), (ValueError, "num_rows", dict(row_indptr=i32(0, 1, 2))),
            (ValueError, "row_indptr", dict(row_indptr=i32(0, 1), num_rows=3)), (ValueError, "at least", dict(num_rows=1)),
            (ValueError, "go together", dict(prefix_pages=pages)), (ValueError, "go together", dict(prefix_lengths=lengths)),
            (ValueError, "several", dict(prefix_pages=pages, prefix_lengths=lengths)),
            (ValueError, "prefix_indptr", dict(prefix_indptr=i32(0, 2))),
            (ValueError, "prefix_pages must", dict(prefix_pages=pages, prefix_lengths=i32(3)))):
        with pytest.raises(kind, match=match):
            plan(**args)
    p, q = plan(), torch.zeros(2, 4, 64, device=DEV).half()
    call = lambda q=q, c=cache, p=p, **kw: sg.prefix_attention(q, c, p, **kw)
    assert not bool(call().any())
    for kind, match, args in (
            (TypeError, "plan", dict(p=None)), (TypeError, "cache", dict(c=None)), (ValueError, "q must", dict(q=q[:1])),
            (TypeError, "q must", dict(q=q.float())), (ValueError, "dense", dict(q=q.new_zeros(2, 4, 128)[..., ::2])),
            (ValueError, "scale", dict(scale=0.0)), (ValueError, "scale", dict(scale=float("inf"))),
            (ValueError, "scale", dict(scale=float("nan"))), (ValueError, "out must", dict(out=q[:1])),
            (ValueError, "lse must", dict(lse=torch.zeros(2, 3, device=DEV))),
            (TypeError, "lse must", dict(lse=torch.zeros(2, 4, device=DEV).half())),
            (ValueError, "other sizes", dict(c=sg.kv_cache(4, 16, 4, 64, torch.float16, device=DEV)))):
        with pytest.raises(kind, match=match):
            call(**args)
    with pytest.raises(RuntimeError, match="no gradients"):
        call(q=q.clone().requires_grad_())
