"""A decoder layer's attention around a quantized cache, as timed workloads.

Three operators, each in its plain form (elementary torch operations in 32
bits) and, with ``own = True``, as the calls a user makes of the library:

  qk_norm_rope      every head of q and k normed, weighted and turned by its
                    position; with its gradients in training
  kv_write, kv_read a paged cache of K and V in 8 or 4 bits, written by slots
                    and read back
  prefix_attention  attention of a batch over such a cache: runs of sequences
                    share a long prefix, every sequence has tokens of its own

A case is a dict of plain values; ``op`` names the operator.
"""
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-6


def _norm(name, R, Hq, Hk, D, rot, layout, dt, far, train):
    return {"name": name, "op": "norm", "rows": R, "q_heads": Hq, "k_heads": Hk, "head_dim": D,
            "rotary_dim": rot, "layout": layout, "dtype": dt, "far": far, "train": train}


def _cache(name, T, Hk, D, page, kind, dt, scattered):
    return {"name": name, "op": "cache", "tokens": T, "k_heads": Hk, "head_dim": D, "page": page,
            "kind": kind, "dtype": dt, "scattered": scattered}


def _attn(name, S, rows, own_lo, own_hi, prefix, groups, Hq, Hk, D, page, kind, dt, mix):
    """S sequences with 1 to ``rows`` new rows and own_lo to own_hi tokens of their own (these
    rows among them), in ``groups`` runs that share about ``prefix`` tokens each."""
    return {"name": name, "op": "attn", "seqs": S, "rows": rows, "own_lo": own_lo, "own_hi": own_hi,
            "prefix": prefix, "groups": groups, "q_heads": Hq, "k_heads": Hk, "head_dim": D,
            "page": page, "kind": kind, "dtype": dt, "mix": mix}


def listed():
    return [
        # One request generating: its q and k, far into a long context.
        _norm("norm_token", 1, 32, 8, 128, 128, "half", "bf16", True, False),
        # A prompt.
        _norm("norm_prompt", 4096, 32, 8, 128, 128, "half", "f16", False, False),
        # A training batch of ragged length, forward and all gradients.
        _norm("norm_train", 8191, 16, 4, 128, 128, "half", "bf16", False, True),
        # A small model of odd sizes in float32, partial interleaved rotation.
        _norm("norm_odd", 1003, 5, 5, 80, 32, "interleaved", "f32", False, True),
        # A decode batch: one new token per sequence, each in a page of its own.
        _cache("cache_decode", 48, 8, 128, 16, "fp8", "bf16", True),
        # A long prompt, into pages wherever they are free, 4 bits.
        _cache("cache_prompt", 8000, 8, 128, 64, "fp4", "f16", False),
        # Ragged rows with padding among them, odd heads, float32.
        _cache("cache_odd", 777, 3, 80, 32, "fp8", "f32", False),
        # A few short requests behind a short instruction.
        _attn("attn_small", 3, 1, 1, 40, 200, 1, 8, 2, 64, 16, "fp8", "f16", 1),
        # A decode batch behind one long document.
        _attn("attn_decode", 64, 1, 64, 1200, 16384, 1, 32, 8, 128, 64, "fp8", "bf16", 2),
        # A decode batch of a model whose heads share nothing, 4-bit cache.
        _attn("attn_decode_4bit", 24, 1, 1, 2000, 6000, 1, 40, 40, 128, 32, "fp4", "f16", 3),
        # Prompts of ragged length behind a common instruction.
        _attn("attn_prompt", 5, 700, 700, 1500, 2048, 1, 32, 8, 128, 64, "fp8", "bf16", 4),
        # Several candidate tokens a sequence, four instructions (one per run), float32.
        _attn("attn_groups", 40, 5, 5, 300, 900, 4, 12, 4, 96, 16, "fp8", "f32", 5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "cache", "attn", "attn", "attn"])
    dt = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
    D = rng.choice([64, 64, 80, 96, 112, 128, 128, 128, 192, 256])
    Hk = rng.choice([1, 2, 3, 4, 8, 8, 16])
    if op == "norm":
        Hq = Hk * rng.choice([1, 2, 4, 5])
        rot = rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)])
        c = _norm(None, _log(rng, 1, 8192), Hq, Hk, D, rot, rng.choice(["half", "interleaved"]), dt,
                  rng.random() < 0.5, rng.random() < 0.5)
        c["rows"] = max(1, min(c["rows"], 2 ** 25 // ((Hq + Hk) * D)))
    elif op == "cache":
        c = _cache(None, _log(rng, 1, 8192), Hk, D, rng.choice([16, 32, 48, 64, 128]),
                   rng.choice(["fp8", "fp4"]), dt, rng.random() < 0.4)
        c["tokens"] = max(1, min(c["tokens"], 2 ** 23 // (Hk * D)))
    else:
        Hq = Hk * rng.choice([1, 2, 4, 4, 7])
        S = _log(rng, 1, 96)
        rows = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 16, 600)])
        hi = rows + _log(rng, 1, 1500)
        c = _attn(None, S, rows, rng.choice([rows, hi // 2 + 1]), hi, rng.choice([0, _log(rng, 16, 16384)]),
                  rng.choice([1, 1, rng.randint(1, 5)]), Hq, Hk, D, rng.choice([16, 32, 48, 64, 128]),
                  rng.choice(["fp8", "fp8", "fp4"]), dt, rng.randrange(10 ** 6))
        c["own_lo"] = max(c["own_lo"], rows)
        limit = 2 ** 34 if dt != "f32" else 2 ** 32
        while work(c)["flops"] > limit or work(c)["bytes"] > 2 ** 27:
            c["seqs"], c["rows"] = (c["seqs"] + 1) // 2, (c["rows"] + 1) // 2
            c["prefix"], c["own_hi"] = c["prefix"] * 3 // 4, max(c["rows"], c["own_hi"] * 3 // 4)
            c["own_lo"] = max(c["rows"], min(c["own_lo"], c["own_hi"]))
    del c["name"]
    return c


# -- the batch of an attention case ---------------------------------------------

def _batch(case):
    """(rows of every sequence, own tokens of every sequence, first sequence of every
    run and the end, prefix tokens of every run)."""
    rng = random.Random(case["mix"])
    S, G = case["seqs"], min(case["groups"], case["seqs"])
    rows = [1 if case["rows"] == 1 else rng.randint(1, case["rows"]) for _ in range(S)]
    tokens = [max(r, rng.randint(case["own_lo"], case["own_hi"])) for r in rows]
    cuts = [0] + sorted(rng.sample(range(1, S), G - 1)) + [S]
    P = case["prefix"]
    prefix = [P if G == 1 else rng.randint(P // 2, P + P // 2) for _ in range(G)]
    return rows, tokens, cuts, prefix


def _running(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


# -- inputs ---------------------------------------------------------------------

def _frequencies(case):
    return 10000.0 ** (-torch.arange(0, case["rotary_dim"], 2, dtype=torch.float64, device="cuda")
                       / case["rotary_dim"])


def _keys_values(gen, T, H, D, dt):
    """Keys with a few strong channels, values of unit variance."""
    k = torch.randn(T, H, D, generator=gen, device="cuda")
    k[..., torch.randperm(D, generator=gen, device="cuda")[: max(1, D // 32)]] *= 4.0
    v = torch.randn(T, H, D, generator=gen, device="cuda")
    return k.to(_DT[dt]), v.to(_DT[dt])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    st = {"case": case}
    if own:
        import segmented_gather_gemv_sgmv_amd as sg
    dt, D, Hk = case["dtype"], case["head_dim"], case["k_heads"]
    if case["op"] == "norm":
        R, Hq = case["rows"], case["q_heads"]
        # q and k are views of the fused projection's output (q, k and v heads)
        qkv = torch.randn(R, Hq + 2 * Hk, D, generator=gen, device="cuda").to(_DT[dt])
        st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        for n in ("wq", "wk"):
            st[n] = (1 + 0.3 * torch.randn(D, generator=gen, device="cuda")).to(_DT[dt])
        top = 100000 if case["far"] else 4096
        if R <= 256:  # a decode batch: every request somewhere of its own
            st["pos"] = torch.randint(0, top, (R,), generator=gen, device="cuda")
        else:  # prompts one after the other
            st["pos"] = (torch.arange(R, device="cuda") + top // 3) % top
        st["freq"] = _frequencies(case)
        if case["train"]:
            st["dq"] = torch.randn(R, Hq, D, generator=gen, device="cuda").to(_DT[dt])
            st["dk"] = torch.randn(R, Hk, D, generator=gen, device="cuda").to(_DT[dt])
        if own:
            st["plan"] = sg.rope_plan(case["rotary_dim"], layout=case["layout"], device="cuda")
            if case["train"]:
                for n in ("q", "k", "wq", "wk"):
                    st[n] = st[n].detach().requires_grad_()
        return st

    page, kind = case["page"], case["kind"]
    if case["op"] == "cache":
        T = case["tokens"]
        st["k"], st["v"] = _keys_values(gen, T, Hk, D, dt)
        if case["scattered"]:  # one token per page, anywhere in it
            pages = T + 5
            at = torch.randperm(pages, generator=gen, device="cuda")[:T] * page
            st["slots"] = at + torch.randint(0, page, (T,), generator=gen, device="cuda")
        else:  # consecutive tokens of a prompt, from the middle of a page on
            first = page // 2 + 1
            pages = (first + T + page - 1) // page + 3
            table = torch.randperm(pages, generator=gen, device="cuda")
            t = torch.arange(T, device="cuda") + first
            st["slots"] = table[t // page] * page + t % page
        if T > 500:  # rows of padding
            st["slots"][torch.randperm(T, generator=gen, device="cuda")[: T // 100]] = -1
        # Read back without the padding.
        st["read"] = st["slots"][st["slots"] >= 0].contiguous()
        st["pages"] = pages
        if own:
            st["cache"] = sg.kv_cache(pages, page, Hk, D, _DT[dt], kind)
        else:
            st["cache"] = _plain_cache(pages * page, Hk, D, kind)
        return st

    rows, tokens, cuts, prefix = _batch(case)
    Hq, T = case["q_heads"], sum(rows)
    st["q"] = (torch.randn(T, Hq, D, generator=gen, device="cuda") * 1.5).to(_DT[dt])
    # Pages of the prefixes and then of the sequences, wherever they are free.
    need = [-(-n // page) for n in prefix + tokens]
    ids = torch.randperm(sum(need) + 3, generator=gen, device="cuda").int()
    first = _running(need)
    width = lambda part: max(1, max(part))
    G = len(prefix)
    st["prefix_pages"] = torch.zeros(G, width(need[:G]), dtype=torch.int32, device="cuda")
    st["own_pages"] = torch.zeros(len(rows), width(need[G:]), dtype=torch.int32, device="cuda")
    slots = []
    for i, n in enumerate(prefix + tokens):
        table = ids[first[i]:first[i + 1]]
        (st["prefix_pages"][i] if i < G else st["own_pages"][i - G])[: need[i]] = table
        t = torch.arange(n, device="cuda")
        slots.append(table[t // page].long() * page + t % page)
    slots = torch.cat(slots)
    k, v = _keys_values(gen, slots.numel(), Hk, D, dt)
    number = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    st["lengths"], st["prefix_lengths"] = number(tokens), number(prefix)
    st["row_indptr"], st["prefix_indptr"] = number(_running(rows)), number(cuts)
    if own:
        st["cache"] = sg.kv_cache(ids.numel(), page, Hk, D, _DT[dt], kind)
        sg.kv_write(st["cache"], k, v, slots)
        # Once per step of the whole model: every layer's call takes it.
        st["plan"] = sg.prefix_plan(
            st["cache"], Hq, st["own_pages"], st["lengths"],
            row_indptr=None if case["rows"] == 1 else st["row_indptr"], num_rows=T,
            prefix_pages=st["prefix_pages"], prefix_lengths=st["prefix_lengths"],
            prefix_indptr=st["prefix_indptr"])
    else:
        st["cache"] = _plain_cache(ids.numel() * page, Hk, D, kind)
        _plain_write(st["cache"], k, v, slots, kind, dt)
        st["k"], st["v"] = k, v  # the prefixes' and then the sequences' tokens
    return st


# -- one pass ---------------------------------------------------------------------

def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    import segmented_gather_gemv_sgmv_amd as sg
    case = st["case"]
    if case["op"] == "norm":
        q, k = sg.qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], st["pos"], st["plan"], eps=_EPS)
        if not case["train"]:
            return [q, k]
        return [q.detach(), k.detach(),
                *torch.autograd.grad([q, k], [st["q"], st["k"], st["wq"], st["wk"]],
                                     [st["dq"], st["dk"]])]
    if case["op"] == "cache":
        sg.kv_write(st["cache"], st["k"], st["v"], st["slots"])
        return list(sg.kv_read(st["cache"], st["read"]))
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float32, device=st["q"].device)
    return [sg.prefix_attention(st["q"], st["cache"], st["plan"], lse=lse), lse]


def _turn(x, cos, sin, case, back):
    """Pairs turned by their angle, or back by it."""
    out, rot = x.clone(), case["rotary_dim"]
    if case["layout"] == "half":
        i, j = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        i, j = slice(0, rot, 2), slice(1, rot, 2)
    a, b = x[..., i], x[..., j]
    if back:
        sin = -sin
    out[..., i] = a * cos - b * sin
    out[..., j] = b * cos + a * sin
    return out


# Largest code, exponent range of the scales (by the cache's type), elements per scale.
_KIND = {"fp8": (448.0, {"bf16": (-116, 119), "f32": (-116, 119), "f16": (-15, 7)}),
         "fp4": (6.0, {"bf16": (-124, 125), "f32": (-124, 125), "f16": (-23, 13)})}


def _plain_cache(slots, H, D, kind):
    """Codes (4 bits: twice the value they stand for) and exponents, by slots."""
    groups = 1 if kind == "fp8" else -(-D // 32)
    codes = torch.zeros(slots, H, D, device="cuda",
                        dtype=torch.float8_e4m3fn if kind == "fp8" else torch.int8)
    return {"k": codes, "v": codes.clone(),
            "ke": torch.zeros(slots, H, groups, dtype=torch.int16, device="cuda"),
            "ve": torch.zeros(slots, H, groups, dtype=torch.int16, device="cuda")}


def _grouped(x, kind):
    """x [..., D] as [..., groups, elements], padded with zeros."""
    if kind == "fp8":
        return x[..., None, :]
    D = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -D % 32))
    return x.reshape(*x.shape[:-1], -1, 32)


def _times(x, e):
    """x 2^e, the power from its bits."""
    return x * ((e.int() + 127) << 23).view(torch.float32)


def _quantize(x, kind, dt):
    """Codes' values [T, H, D] (float32) and exponents [T, H, groups]."""
    D, (most, limits) = x.shape[-1], _KIND[kind]
    lo, hi = limits[dt]
    g = _grouped(x.float(), kind)
    size = g.abs().amax(-1)
    # least e with size <= most 2^e: most = 0.875 2^9 or 0.75 2^3
    frac, e = torch.frexp(size)
    part, top = math.frexp(most)
    e = (e - top + (frac > part)).clamp(lo, hi)
    e = torch.where(size == 0, torch.full_like(e, lo), e)
    y = _times(g, -e[..., None]).clamp(-most, most)
    # round to 3 bits behind the first (4-bit codes: 1), less where the exponent ends
    bits, least = (3, -6) if kind == "fp8" else (1, 0)
    exponent = (torch.frexp(y)[1] - 1).clamp(min=least)
    y = _times(torch.round(_times(y, bits - exponent)), exponent - bits)
    return y.flatten(-2)[..., :D], e


def _plain_write(cache, k, v, slots, kind, dt):
    held = slots >= 0
    for n, x in (("k", k), ("v", v)):
        y, e = _quantize(x, kind, dt)
        y = y.to(torch.float8_e4m3fn) if kind == "fp8" else (2 * y).to(torch.int8)
        cache[n].view(torch.int8)[slots[held]] = y.view(torch.int8)[held]
        cache[n + "e"][slots[held]] = e.to(torch.int16)[held]


def _plain_read(cache, slots, kind):
    """k and v of the slots in float32."""
    out = []
    for n in ("k", "v"):
        codes = cache[n].view(torch.int8)[slots]
        y = codes.view(torch.float8_e4m3fn).float() if kind == "fp8" else codes.float() / 2
        g = _times(_grouped(y, kind), cache[n + "e"][slots][..., None])
        out.append(g.flatten(-2)[..., : y.shape[-1]])
    return out


def _tables(st):
    """Slots of every prefix's and every sequence's tokens."""
    case = st["case"]
    rows, tokens, cuts, prefix = _batch(case)
    page = case["page"]

    def slots(table, n):
        t = torch.arange(n, device="cuda")
        return table[t // page].long() * page + t % page

    return (rows, tokens, cuts, prefix,
            [slots(st["prefix_pages"][g], n) for g, n in enumerate(prefix)],
            [slots(st["own_pages"][i], n) for i, n in enumerate(tokens)])


def _part(q, k, v, scale, visible):
    """Sum of exp(s - m) v, sum of exp(s - m) and m of rows [N, Hq, D] over keys [n, Hk, D];
    visible [N] counts the keys that a row sees (None: all)."""
    N, Hq, D = q.shape
    n, Hk, _ = k.shape
    q = q.reshape(N, Hk, Hq // Hk, D).permute(1, 0, 2, 3).reshape(Hk, -1, D).contiguous()
    s = torch.matmul(q, k.permute(1, 2, 0).contiguous()) * scale
    s = s.view(Hk, N, Hq // Hk, n)
    if visible is not None:
        hidden = torch.arange(n, device=q.device)[None, :] >= visible[:, None]
        s = s.masked_fill(hidden[None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    o = torch.matmul(p.view(Hk, -1, n), v.permute(1, 0, 2).contiguous())
    back = lambda t: t.reshape(Hk, N, Hq // Hk, -1).permute(1, 0, 2, 3).reshape(N, Hq, -1)
    return back(o), back(p.sum(-1, keepdim=True)), back(m)


def _attend(st):
    case = st["case"]
    rows, tokens, cuts, prefix, prefix_slots, own_slots = _tables(st)
    scale, kind = 1 / math.sqrt(case["head_dim"]), case["kind"]
    q, first, parts = st["q"].float(), _running(rows), []
    for i, (n, length) in enumerate(zip(rows, tokens)):
        k, v = _plain_read(st["cache"], own_slots[i], kind)
        visible = None if n == 1 else torch.arange(length - n + 1, length + 1, device=q.device)
        parts.append(_part(q[first[i]:first[i + 1]], k, v, scale, visible))
    o, l, m = (torch.cat(t) for t in zip(*parts))
    if sum(prefix):
        held = []
        for g, n in enumerate(prefix):  # once for all sequences of a run
            k, v = _plain_read(st["cache"], prefix_slots[g], kind)
            held.append(_part(q[first[cuts[g]]:first[cuts[g + 1]]], k, v, scale, None))
        po, pl, pm = (torch.cat(t) for t in zip(*held))
        top = torch.maximum(m, pm)
        a, b = torch.exp(m - top), torch.exp(pm - top)
        o, l, m = a * o + b * po, a * l + b * pl, top
    return [(o / l).to(_DT[case["dtype"]]), (m + torch.log(l))[..., 0]]


def _plain(st):
    case = st["case"]
    dt = _DT[case["dtype"]]
    if case["op"] == "attn":
        return _attend(st)
    if case["op"] == "cache":
        _plain_write(st["cache"], st["k"], st["v"], st["slots"], case["kind"], case["dtype"])
        return [t.to(dt) for t in _plain_read(st["cache"], st["read"], case["kind"])]
    angle = st["pos"].double()[:, None] * st["freq"][None, :]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out, grads, weights = [], [], []
    for n in ("q", "k"):
        x, w = st[n].float(), st["w" + n].float()
        r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS)
        out.append(_turn(x * r * w, cos, sin, case, False).to(dt))
        if case["train"]:
            dn = _turn(st["d" + n].float(), cos, sin, case, True)
            weights.append((dn * x * r).sum((0, 1)).to(dt))
            dn = dn * w
            grads.append((r * (dn - x * r * r * (dn * x).mean(-1, keepdim=True))).to(dt))
    return out + grads + weights


# -- the definition in 64 bits -----------------------------------------------------

def _exact_norm(st, case):
    rot = case["rotary_dim"]
    angle = st["pos"].double()[:, None] * st["freq"][None, :]
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    with torch.enable_grad():
        leaves = [st[n].double().requires_grad_(case["train"]) for n in ("q", "k", "wq", "wk")]
        out = []
        for x, w in zip(leaves[:2], leaves[2:]):
            y = w * x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)
            if case["layout"] == "half":
                z = torch.complex(y[..., : rot // 2], y[..., rot // 2: rot]) * turn
                y = torch.cat([z.real, z.imag, y[..., rot:]], -1)
            else:
                pairs = y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2)
                z = torch.complex(pairs[..., 0], pairs[..., 1]) * turn
                y = torch.cat([torch.stack([z.real, z.imag], -1).flatten(-2), y[..., rot:]], -1)
            out.append(y)
        if not case["train"]:
            return out
        grads = torch.autograd.grad(out, leaves, [st["dq"].double(), st["dk"].double()])
    return [t.detach() for t in out] + list(grads)


def _nearest(x, kind, dt):
    """The value that a cache keeps of x, by looking every code up."""
    most, limits = _KIND[kind]
    lo, hi = limits[dt]
    if kind == "fp8":  # 0, 1/8 .. 7/8 times 2^-6, then 8/8 .. 15/8 times 2^-6 .. 2^8, but for the last
        grid = [m / 8 * 2.0 ** -6 for m in range(8)]
        grid += [(8 + m) / 8 * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1]
        group = x.shape[-1]
    else:
        grid, group = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], 32
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    between = (grid[1:] + grid[:-1]) / 2
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for at in range(0, x.shape[-1], group):
        part = x[..., at: at + group].double()
        size = part.abs().amax(-1, keepdim=True)
        e = torch.full_like(size, lo)
        for step in range(lo, hi):
            e += (size > most * 2.0 ** step).double()
        y = (part.abs() * torch.exp2(-e)).clamp(max=most)
        code = torch.bucketize(y, between)  # a tie goes down ...
        tie = (code < between.numel()) & (y == between[code.clamp(max=between.numel() - 1)])
        code = code + (tie & (code % 2 == 1)).long()  # ... or to the even code
        out[..., at: at + group] = grid[code] * part.sign() * torch.exp2(e)
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "norm":
        return _exact_norm(st, case)
    if case["op"] == "cache":
        keep = st["slots"] >= 0
        return [_nearest(st[n][keep], case["kind"], case["dtype"]) for n in ("k", "v")]
    rows, tokens, cuts, prefix = _batch(case)
    at = _running(prefix + tokens)
    held = [_nearest(st[n], case["kind"], case["dtype"]) for n in ("k", "v")]
    Hq, Hk, D = case["q_heads"], case["k_heads"], case["head_dim"]
    first, outs, lses = _running(rows), [], []
    for i, (n, length) in enumerate(zip(rows, tokens)):
        g = max(j for j in range(len(prefix)) if cuts[j] <= i)
        j = len(prefix) + i
        k, v = (torch.cat([t[at[g]:at[g + 1]], t[at[j]:at[j + 1]]]) for t in held)
        q = st["q"][first[i]:first[i + 1]].double()
        last = prefix[g] + length - n + torch.arange(n, device=q.device)
        seen = torch.arange(k.shape[0], device=q.device)[None, :] <= last[:, None]
        o, lse = torch.empty_like(q), q.new_empty(n, Hq)
        for h in range(Hq):
            c = h // (Hq // Hk)
            s = torch.where(seen, torch.mm(q[:, h], k[:, c].t()) / math.sqrt(D), -math.inf)
            lse[:, h] = torch.logsumexp(s, 1)
            o[:, h] = torch.mm(torch.softmax(s, 1), v[:, c])
        outs.append(o)
        lses.append(lse)
    return [torch.cat(outs), torch.cat(lses)]


# -- what a pass cannot do without ---------------------------------------------------

def work(case):
    b, D, Hk = _BYTES[case["dtype"]], case["head_dim"], case["k_heads"]
    if case["op"] == "norm":
        heads = case["q_heads"] + Hk
        n = case["rows"] * heads * D
        turned = case["rows"] * heads * case["rotary_dim"]
        if not case["train"]:
            return {"bytes": 2 * n * b + 8 * case["rows"] + 2 * D * b, "flops": 5 * n + 3 * turned}
        # forward: x in, y out; backward: x and dy in, dx out
        return {"bytes": 5 * n * b + 16 * case["rows"] + 6 * D * b, "flops": 15 * n + 6 * turned}
    groups = 1 if case["kind"] == "fp8" else -(-D // 32)
    held = Hk * (D * (8 if case["kind"] == "fp8" else 4) / 8 + groups)  # of a token, K or V
    if case["op"] == "cache":
        n = 2 * case["tokens"] * Hk * D
        return {"bytes": int(2 * n * b + 4 * case["tokens"] * held) + 16 * case["tokens"],
                "flops": 4 * n}
    rows, tokens, cuts, prefix = _batch(case)
    first = _running(rows)
    pairs = sum((first[cuts[g + 1]] - first[cuts[g]]) * p for g, p in enumerate(prefix))
    pairs += sum(n * (length - n) + n * (n + 1) // 2 for n, length in zip(rows, tokens))
    Hq = case["q_heads"]
    return {"bytes": int(2 * held * (sum(prefix) + sum(tokens))) + sum(rows) * Hq * (2 * D * b + 4),
            "flops": 4 * pairs * Hq * D}
