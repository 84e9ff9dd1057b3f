"""The projections around a multi-LoRA decoder layer, as timed workloads.

Four operators, each in its plain form (elementary torch operations in 32
bits) and, with ``own = True``, as the calls a user makes of the library:

  q4_linear     y = x W^T + b with 4-bit weight codes, one scale (and zero
                point) per group of G input columns
  q4_gated_ffn  h = act(x Wg^T + a_g) * (x Wu^T + a_u), both weights 4-bit
  gated_ffn     the same with float weights; with its gradients in training
  rope          rotary positions on q and k; with its gradients in training

A case is a dict of plain values; ``op`` names the operator.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def _q4(name, R, H1, H2, G, dt, zeros, bias):
    return {"name": name, "op": "q4_linear", "rows": R, "in": H1, "out": H2, "group": G,
            "dtype": dt, "zeros": zeros, "bias": bias}


def _q4g(name, R, H1, I, G, dt, zeros, act, add):
    return {"name": name, "op": "q4_gated_ffn", "rows": R, "in": H1, "out": I, "group": G,
            "dtype": dt, "zeros": zeros, "act": act, "add": add}


def _ffn(name, R, H, I, dt, act, train, add, frozen):
    return {"name": name, "op": "gated_ffn", "rows": R, "in": H, "out": I, "dtype": dt, "act": act,
            "train": train, "add": add, "frozen": frozen}


def _rope(name, R, Hq, Hk, D, rot, layout, dt, scaling, far, train):
    return {"name": name, "op": "rope", "rows": R, "q_heads": Hq, "k_heads": Hk, "head_dim": D,
            "rotary_dim": rot, "layout": layout, "dtype": dt, "scaling": scaling, "far": far,
            "train": train}


def listed():
    return [
        # One request generating: an attention projection of a 7B model.
        _q4("q4_token", 1, 4096, 4096, 128, "f16", False, False),
        # A decode batch through a 13B model's up projection.
        _q4("q4_decode", 24, 5120, 13824, 64, "bf16", True, False),
        # A prompt of ragged length through an attention projection with a bias.
        _q4("q4_prefill", 1531, 4096, 4096, 128, "bf16", True, True),
        # A small head of odd sizes in float32, ragged last group.
        _q4("q4_odd", 5, 1000, 333, 32, "f32", True, True),
        # A few adapted requests generating: a 7B model's gate and up projections.
        _q4g("q4_gated_decode", 7, 4096, 11008, 128, "bf16", False, "silu", True),
        # A chunk of prompt through the same block of a smaller model.
        _q4g("q4_gated_chunk", 333, 2048, 5632, 32, "f16", True, "gelu_tanh", False),
        # One request generating with 16-bit weights.
        _ffn("ffn_token", 1, 4096, 11008, "bf16", "silu", False, False, False),
        # A prompt.
        _ffn("ffn_prefill", 2048, 4096, 11008, "f16", "silu", False, False, False),
        # Full fine-tuning step of the block, forward and all gradients.
        _ffn("ffn_train", 4096, 4096, 11008, "bf16", "silu", True, False, False),
        # Adapter fine-tuning on a ragged batch: the base weights are frozen, the
        # adapters' addends and x get gradients.
        _ffn("ffn_adapter_train", 1237, 1000, 2744, "f16", "gelu_tanh", True, True, True),
        # A decode batch's q and k, far into a scaled long context.
        _rope("rope_decode", 64, 32, 32, 128, 128, "half", "bf16", "by_parts", True, False),
        # A training batch with partial interleaved rotation, and its gradients.
        _rope("rope_train", 8191, 32, 8, 80, 32, "interleaved", "bf16", "none", False, True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["q4_linear", "q4_linear", "q4_gated_ffn", "gated_ffn", "gated_ffn", "rope"])
    dt = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
    act = rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 192, 256])
        rot = rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)])
        Hk = rng.choice([1, 2, 4, 8, 32])
        Hq = Hk * rng.choice([1, 3, 4, 7]) if Hk < 32 else 32
        c = _rope(None, _log(rng, 1, 8192), Hq, Hk, D, rot, rng.choice(["half", "interleaved"]), dt,
                  rng.choice(["none", "linear", "ntk", "by_parts"]), rng.random() < 0.5,
                  rng.random() < 0.4)
        if c["rows"] * (Hq + Hk) * D > 2 ** 27:
            c["rows"] = 2 ** 27 // ((Hq + Hk) * D)
    elif op == "gated_ffn":
        if rng.random() < 0.1:  # sizes that fit no vector
            H, I, R = _log(rng, 65, 600) | 1, _log(rng, 65, 600) | 1, _log(rng, 1, 300)
        else:
            H, I = _log(rng, 256, 4096, 8), _log(rng, 512, 11008, 8)
            R = _log(rng, 1, 4096 if dt != "f32" else 512)
        train = R >= 32 and rng.random() < 0.6
        c = _ffn(None, R, H, I, dt, act, train, rng.random() < 0.4, train and rng.random() < 0.4)
    else:
        if rng.random() < 0.1:
            H1, H2, R = _log(rng, 33, 900) | 1, _log(rng, 33, 900) | 1, _log(rng, 1, 300)
        else:
            H1, H2 = _log(rng, 256, 8192, 8), _log(rng, 256, 13824, 8)
            R = _log(rng, 1, 2048 if dt != "f32" else 256)
        G = rng.choice([32, 64, 128])
        if op == "q4_linear":
            c = _q4(None, R, H1, H2, G, dt, rng.random() < 0.5, rng.random() < 0.5)
        else:
            c = _q4g(None, R, H1, H2, G, dt, rng.random() < 0.5, act, rng.random() < 0.5)
    del c["name"]
    return c


# -- inputs ------------------------------------------------------------------

def _activations(gen, R, H, dt):
    """Normed hidden states: unit variance, a few channels much larger."""
    x = torch.randn(R, H, generator=gen, device="cuda")
    big = torch.randperm(H, generator=gen, device="cuda")[: max(1, H // 512)]
    x[:, big] *= 8.0
    return x.to(_DT[dt])


def _quantized(gen, n, k, G, dt, zeros):
    """Codes [n, ceil(k / 2)] (column 2 j in the low half of byte j), scales
    [n, groups] and zero points of a normal weight rounded to nearest."""
    ng = (k + G - 1) // G
    w = torch.randn(n, ng * G, generator=gen, device="cuda") * (0.7 / math.sqrt(k))
    w = w.view(n, ng, G)
    if zeros:
        lo, hi = w.amin(2), w.amax(2)
        s = ((hi - lo) / 15).to(_DT[dt])
        z = (-lo / s.float()).round().clamp(0, 15)
    else:
        s = (w.abs().amax(2) / 7.5).to(_DT[dt])
        z = torch.full((n, ng), 8.0, device="cuda")
    q = (w / s.float()[..., None] + z[..., None]).round().clamp(0, 15)
    q = q.view(n, ng * G)[:, :k].to(torch.uint8)
    if k % 2:
        q = torch.cat([q, q.new_zeros(n, 1)], 1)
    codes = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    return codes, s.contiguous(), z.to(torch.uint8).contiguous() if zeros else None


def _scaled_frequencies(case):
    """inv_freq [rot / 2] (float64, on the host) and the magnitude factor."""
    rot, base = case["rotary_dim"], 10000.0
    factor, ctx = 8.0, 4096
    j = torch.arange(0, rot, 2, dtype=torch.float64)
    if case["scaling"] == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-j / rot)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "by_parts":
        # Frequencies that turn often within the trained context stay, those
        # that turn less than once are interpolated, a ramp between.
        def dim(turns):
            return rot * math.log(ctx / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    op, dt, R = case["op"], case["dtype"], case["rows"]
    st = {"case": case}
    if op == "rope":
        Hq, Hk, D = case["q_heads"], case["k_heads"], case["head_dim"]
        # q and k are views of the fused projection's output (q, k and v heads)
        qkv = torch.randn(R, Hq + 2 * Hk, D, generator=gen, device="cuda").to(_DT[dt])
        st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        top = 32768 if case["far"] else 4096
        if R <= 256:  # a decode batch: every request somewhere of its own
            st["pos"] = torch.randint(0, top, (R,), generator=gen, device="cuda")
        else:  # prompts one after the other
            st["pos"] = (torch.arange(R, device="cuda") + top // 3) % top
        st["freq"], st["mag"] = _scaled_frequencies(case)
        st["freq"] = st["freq"].cuda()
        if case["train"]:
            st["dq"] = torch.randn(R, Hq, D, generator=gen, device="cuda").to(_DT[dt])
            st["dk"] = torch.randn(R, Hk, D, generator=gen, device="cuda").to(_DT[dt])
        if own:
            import segmented_gather_gemv_sgmv_amd as sg
            scaling = {"none": None, "linear": {"kind": "linear", "factor": 8.0},
                       "ntk": {"kind": "ntk", "factor": 8.0},
                       "by_parts": {"kind": "by_parts", "factor": 8.0, "context": 4096}}
            st["plan"] = sg.rope_plan(case["rotary_dim"], base=10000.0,
                                      scaling=scaling[case["scaling"]], layout=case["layout"],
                                      device="cuda")
            if case["train"]:
                st["q"] = st["q"].detach().requires_grad_()
                st["k"] = st["k"].detach().requires_grad_()
        return st
    H, N = case["in"], case["out"]
    st["x"] = _activations(gen, R, H, dt)
    if op == "q4_linear":
        st["w"] = _quantized(gen, N, H, case["group"], dt, case["zeros"])
        st["bias"] = (torch.randn(N, generator=gen, device="cuda") * 0.1).to(_DT[dt]) \
            if case["bias"] else None
    elif op == "q4_gated_ffn":
        st["g"] = _quantized(gen, N, H, case["group"], dt, case["zeros"])
        st["u"] = _quantized(gen, N, H, case["group"], dt, case["zeros"])
    else:
        s = 0.7 / math.sqrt(H)
        st["Wg"] = (torch.randn(N, H, generator=gen, device="cuda") * s).to(_DT[dt])
        st["Wu"] = (torch.randn(N, H, generator=gen, device="cuda") * s).to(_DT[dt])
        if case["train"]:
            st["dh"] = (torch.randn(R, N, generator=gen, device="cuda") * 0.1).to(_DT[dt])
    if case.get("add"):  # what the rows' adapters add before the activation
        st["ag"] = (torch.randn(R, N, generator=gen, device="cuda") * 0.2).to(_DT[dt])
        st["au"] = (torch.randn(R, N, generator=gen, device="cuda") * 0.2).to(_DT[dt])
    else:
        st["ag"] = st["au"] = None
    if own:
        import segmented_gather_gemv_sgmv_amd as sg
        G = case.get("group")
        if op == "q4_linear":
            st["W4"] = sg.q4_pack(*st["w"], group_size=G, in_features=H)
        elif op == "q4_gated_ffn":
            st["G4"] = sg.q4_pack(*st["g"], group_size=G, in_features=H)
            st["U4"] = sg.q4_pack(*st["u"], group_size=G, in_features=H)
        elif case["train"]:
            wants = ["x"] + ([] if case["frozen"] else ["Wg", "Wu"])
            wants += ["ag", "au"] if case["add"] else []
            for n in wants:
                st[n].requires_grad_()
            st["wants"] = [st[n] for n in wants]
    return st


# -- one pass ----------------------------------------------------------------

def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    import segmented_gather_gemv_sgmv_amd as sg
    case = st["case"]
    op = case["op"]
    if op == "q4_linear":
        return sg.q4_linear(st["x"], st["W4"], bias=st["bias"])
    if op == "q4_gated_ffn":
        return sg.q4_gated_ffn(st["x"], st["G4"], st["U4"], act=case["act"], gate_add=st["ag"],
                               up_add=st["au"])
    if op == "gated_ffn":
        h = sg.gated_ffn(st["x"], st["Wg"], st["Wu"], act=case["act"], gate_add=st["ag"],
                         up_add=st["au"])
        if not case["train"]:
            return h
        return [h.detach(), *torch.autograd.grad(h, st["wants"], st["dh"])]
    q, k = sg.rope(st["q"], st["k"], st["pos"], st["plan"])
    if not case["train"]:
        return [q, k]
    return [q.detach(), k.detach(),
            *torch.autograd.grad([q, k], [st["q"], st["k"]], [st["dq"], st["dk"]])]


def _act(name, g):
    """act(g) and its derivative."""
    if name == "relu":
        return g.clamp(min=0), (g > 0).to(g.dtype)
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(g / math.sqrt(2.0)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), \
            0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    s = 1 / (1 + torch.exp(-g))
    if name == "sigmoid":
        return s, s * (1 - s)
    return g * s, s * (1 + g * (1 - s))


def _dequantize(w, k, G):
    """The weight [n, k] in float32."""
    codes, s, z = w
    n = codes.shape[0]
    q = torch.stack([codes & 15, codes >> 4], 2).view(n, -1)[:, :k].float()
    z = z.float().repeat_interleave(G, 1)[:, :k] if z is not None else 8.0
    return (q - z) * s.float().repeat_interleave(G, 1)[:, :k]


def _rotate(x, cos, sin, rot, layout, mag):
    out = x.clone()
    if layout == "half":
        i, j = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        i, j = slice(0, rot, 2), slice(1, rot, 2)
    a, b = x[..., i], x[..., j]
    out[..., i] = (a * cos - b * sin) * mag
    out[..., j] = (b * cos + a * sin) * mag
    return out


def _plain(st):
    case = st["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "rope":
        ang = st["pos"].double()[:, None] * st["freq"][None, :]
        cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
        rot, lay, m = case["rotary_dim"], case["layout"], st["mag"]
        out = [_rotate(st[n].float(), cos, sin, rot, lay, m).to(dt) for n in ("q", "k")]
        if case["train"]:  # the gradients turn back by the same angles
            out += [_rotate(st[n].float(), cos, -sin, rot, lay, m).to(dt) for n in ("dq", "dk")]
        return out
    x = st["x"].float()
    if op == "q4_linear":
        y = x @ _dequantize(st["w"], case["in"], case["group"]).t()
        if st["bias"] is not None:
            y = y + st["bias"].float()
        return y.to(dt)
    if op == "q4_gated_ffn":
        Wg = _dequantize(st["g"], case["in"], case["group"])
        Wu = _dequantize(st["u"], case["in"], case["group"])
    else:
        Wg, Wu = st["Wg"].float(), st["Wu"].float()
    g, u = x @ Wg.t(), x @ Wu.t()
    if st["ag"] is not None:
        g, u = g + st["ag"].float(), u + st["au"].float()
    a, d = _act(case["act"], g)
    h = (a * u).to(dt)
    if not case.get("train"):
        return h
    dh = st["dh"].float()
    dg, du = dh * u * d, dh * a
    out = [h, (dg @ Wg + du @ Wu).to(dt)]
    if not case["frozen"]:
        out += [(dg.t() @ x).to(dt), (du.t() @ x).to(dt)]
    if case["add"]:
        out += [dg.to(dt), du.to(dt)]
    return out


# -- the definition in 64 bits -----------------------------------------------

def _weight64(w, k, G):
    codes, s, z = w
    col = torch.arange(k, device=codes.device)
    q = (codes[:, col // 2] >> (4 * (col % 2)).to(torch.uint8)) & 15
    zero = z[:, col // G].double() if z is not None else 8.0
    return s[:, col // G].double() * (q.double() - zero)


def _act64(name, g):
    with torch.enable_grad():
        t = g.clone().requires_grad_()
        if name == "silu":
            a = t * torch.sigmoid(t)
        elif name == "sigmoid":
            a = torch.sigmoid(t)
        elif name == "relu":
            a = torch.where(t > 0, t, torch.zeros_like(t))
        elif name == "gelu":
            a = t * 0.5 * torch.erfc(-t * math.sqrt(0.5))
        else:
            a = 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))
        return a.detach(), torch.autograd.grad(a.sum(), t)[0]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rope":
        rot, m = case["rotary_dim"], st["mag"]
        ang = st["pos"].double()[:, None] * st["freq"][None, :]
        turn = torch.polar(torch.full_like(ang, m), ang)[:, None]

        def rotated(x, turn):
            y = x.double().clone()
            if case["layout"] == "half":
                z = torch.complex(y[..., : rot // 2], y[..., rot // 2: rot]) * turn
                y[..., :rot] = torch.cat([z.real, z.imag], -1)
            else:
                z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2)) * turn
                y[..., :rot] = torch.view_as_real(z).flatten(-2)
            return y

        out = [rotated(st["q"], turn), rotated(st["k"], turn)]
        if case["train"]:
            out += [rotated(st["dq"], turn.conj()), rotated(st["dk"], turn.conj())]
        return out
    x = st["x"].double()
    if case["op"] == "q4_linear":
        y = torch.mm(x, _weight64(st["w"], case["in"], case["group"]).t())
        return y if st["bias"] is None else y + st["bias"].double()
    if case["op"] == "q4_gated_ffn":
        Wg, Wu = (_weight64(st[n], case["in"], case["group"]) for n in ("g", "u"))
    else:
        Wg, Wu = st["Wg"].double(), st["Wu"].double()
    g, u = torch.mm(x, Wg.t()), torch.mm(x, Wu.t())
    if st["ag"] is not None:
        g += st["ag"].double()
        u += st["au"].double()
    a, d = _act64(case["act"], g)
    if not case.get("train"):
        return a * u
    dh = st["dh"].double()
    dg, du = dh * u * d, dh * a
    out = [a * u, torch.mm(dg, Wg) + torch.mm(du, Wu)]
    if not case["frozen"]:
        out += [torch.mm(dg.t(), x), torch.mm(du.t(), x)]
    if case["add"]:
        out += [dg, du]
    return out


# -- what a pass cannot do without --------------------------------------------

def work(case):
    b, R = _BYTES[case["dtype"]], case["rows"]
    if case["op"] == "rope":
        n = R * (case["q_heads"] + case["k_heads"]) * case["head_dim"]
        passes = 2 if case["train"] else 1
        turned = R * (case["q_heads"] + case["k_heads"]) * case["rotary_dim"]
        return {"bytes": passes * (2 * n * b + 8 * R), "flops": passes * 3 * turned}
    H, N = case["in"], case["out"]
    if case["op"] != "gated_ffn":
        ng = -(-H // case["group"])
        w = N * -(-H // 2) + N * ng * (b + (1 if case["zeros"] else 0))
        if case["op"] == "q4_linear":
            return {"bytes": w + b * (R * H + R * N + (N if case["bias"] else 0)),
                    "flops": 2 * R * H * N}
        return {"bytes": 2 * w + b * (R * H + R * N + (2 * R * N if case["add"] else 0)),
                "flops": 4 * R * H * N}
    nbytes = b * (R * H + 2 * H * N + R * N + (2 * R * N if case["add"] else 0))
    flops = 4 * R * H * N
    if case["train"]:
        nbytes += b * (R * N + R * H)  # dh in, dx out
        flops += 4 * R * H * N
        if not case["frozen"]:
            nbytes += b * 2 * H * N
            flops += 4 * R * H * N
        if case["add"]:
            nbytes += b * 2 * R * N
    return {"bytes": nbytes, "flops": flops}
