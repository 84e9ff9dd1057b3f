"""How prefix_plan cuts a step into items, in plain Python, and what the C ABI reserves for it."""
import ctypes

TARGET, LEAST, KEYS = 448, 6, 64


def widest(padded, dtype):
    """Rows of the widest tile (dtype: 0 float32)."""
    return 128 if padded <= 128 and dtype != 0 else 64


def cut(rows, tokens, cuts, prefix, rep, kv_heads, wide):
    """(items, slots) of sequences with rows[i] rows and tokens[i] tokens, runs of them (cuts) behind
    prefixes."""
    blocks = lambda n: -(-n // KEYS)
    run = [next((g for g in range(len(prefix)) if cuts[g] <= i < cuts[g + 1]), -1) for i in range(len(rows))]
    apart = [any(run[i] == g and 0 < rows[i] * rep < wide for i in range(len(rows))) for g in range(len(prefix))]
    stacks = []  # rows of a K / V head, blocks, whether its rows see nothing else
    for g, n in enumerate(prefix):
        mine = sum(r for r, x in zip(rows, run) if x == g)
        stacks.append((mine * rep if apart[g] else 0, blocks(n), False))
    for r, n, g in zip(rows, tokens, run):
        front = 0 if g < 0 or apart[g] else prefix[g]
        stacks.append((r * rep, blocks(n) + blocks(front), g < 0 or not apart[g] or prefix[g] == 0))
    tile = lambda m: next((t for t in (16, 32, 64, 128) if t >= m and t <= wide), wide)
    weight = lambda m: 2 if tile(m) >= 64 else 1
    tiles = lambda m: -(-m // tile(m))
    work = sum(kv_heads * tiles(m) * b * weight(m) for m, b, _ in stacks)
    chunk = max(LEAST, -(-work // TARGET))
    items = slots = 0
    for m, b, only in stacks:
        if m == 0 or b == 0:
            continue
        chunks = max(1, (10 * b * weight(m) + 3 * chunk) // (10 * chunk))
        items += kv_heads * tiles(m) * chunks
        if not (only and chunks == 1):
            slots += kv_heads * tiles(m) * chunks * tile(m)
    return items, slots


def reserved(lib, cache, rows, seqs, prefixes, q_heads, dtype):
    """(items, slots) that the plan and the workspace have room for, None for sizes that are refused."""
    p, sizes = ctypes.addressof(cache), (rows, seqs, prefixes, q_heads, dtype)
    padded = lib.kv_codes_bytes(1, 16, 1, cache.head_dim, 0) // 16
    ints = lib.prefix_plan_bytes(p, *sizes) // 4
    if ints == 0:
        return None
    items, rest = divmod(ints - 16 - 12 * (seqs + prefixes) - rows - seqs - prefixes, 16)
    slots, left = divmod(lib.prefix_attention_workspace_bytes(p, *sizes), 4 * padded + 8)
    assert rest == 0 and left == 0
    return items, slots


def draw(rng):
    """(rows, tokens, cuts, prefix, rep, kv_heads) of a batch."""
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    S = rng.choice([1, 1, 2, 3, rng.randint(4, 40), log(40, 600)])
    kind = rng.choice(["decode", "prompts", "mixed"])
    top = log(1, 4000)
    rows = [1 if kind == "decode" or (kind == "mixed" and rng.random() < 0.7) else rng.randint(0, top) for _ in range(S)]
    tokens = [rng.choice([0, r, r + log(1, 3000), log(1, 60000)]) for r in rows]
    G = rng.choice([0, 0, 1, 1, rng.randint(1, min(S, 5))])
    cuts = sorted(rng.randint(0, S) for _ in range(G + 1))
    prefix = [rng.choice([0, log(1, 200), log(1, 50000)]) for _ in range(G)]
    return rows, tokens, cuts, prefix, rng.choice([1, 1, 2, 4, 7, 16]), rng.choice([1, 2, 8, 40])
