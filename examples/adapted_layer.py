"""A decoder layer with a 4-bit base and many adapters: one batch served, then
its feed-forward adapters trained.

    python examples/adapted_layer.py

Serving: q, k and v by q4_linear with every row's own adapter added by
lora_apply_multi, rope on q and k, causal attention over the batch (plain
torch: the layer's own operators are what this shows), then the gated block
by q4_gated_ffn with the adapters' addends entering before its activation.
Training: the same block with 16-bit weights, frozen, by gated_ffn; the
gradients of its addends and of x reach the adapters.  Weights are random.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import segmented_gather_gemv_sgmv_amd as sg  # noqa: E402


class AdaptedLayer:
    """Base weights in 4 bits (groups of ``group`` input features, zero points) and a stack of
    ``adapters`` rank-``rank`` adapters on q, v, gate and up."""

    def __init__(self, hidden, ffn, heads, adapters, rank, dtype, group=64, seed=0, device="cuda"):
        self.hidden, self.ffn, self.heads, self.group, self.dtype = hidden, ffn, heads, group, dtype
        gen = torch.Generator().manual_seed(seed)
        self.raw, self.weights, self.lora = {}, {}, {}
        shapes = dict(q=(hidden, hidden), k=(hidden, hidden), v=(hidden, hidden), o=(hidden, hidden),
                      gate=(ffn, hidden), up=(ffn, hidden), down=(hidden, ffn))
        for name, (n, k) in shapes.items():
            groups = -(-k // group)
            raw = (torch.randint(0, 256, (n, (k + 1) // 2), generator=gen, dtype=torch.uint8),
                   ((0.5 + torch.rand(n, groups, generator=gen)) * 0.2 / math.sqrt(k)).to(dtype),
                   torch.randint(6, 10, (n, groups), generator=gen, dtype=torch.uint8))
            self.raw[name] = tuple(t.to(device) for t in raw)
            self.weights[name] = sg.q4_pack(*self.raw[name], group_size=group, in_features=k)
        for name in ("q", "v", "gate", "up"):
            n, k = shapes[name]
            self.lora[name] = tuple((torch.randn(s, generator=gen) / math.sqrt(s[1])).to(dtype).to(device)
                                    for s in ((adapters, k, rank), (adapters, rank, n)))
        self.plan = sg.rope_plan(hidden // heads, scaling={"kind": "linear", "factor": 2.0}, device=device)

    def _adapt(self, x, outputs, segments):
        """Adds every row's adapter to the named outputs, in one launch."""
        seg, ids = segments
        sg.lora_apply_multi([(y, x, *self.lora[name], 1.0) for name, y in outputs.items()], seg, ids)

    def serve(self, x, positions, segments):
        """The layer's output for rows x [R, hidden] of one sequence."""
        R, w = x.shape[0], self.weights
        q, k, v = (sg.q4_linear(x, w[n]) for n in "qkv")
        self._adapt(x, dict(q=q, v=v), segments)
        q, k, v = (t.view(R, self.heads, -1) for t in (q, k, v))
        sg.rope(q, k, positions, self.plan, out=(q, k))
        attended = x + sg.q4_linear(self._attend(q, k, v), w["o"])
        gate = attended.new_zeros(R, self.ffn)
        up = torch.zeros_like(gate)
        self._adapt(attended, dict(gate=gate, up=up), segments)
        h = sg.q4_gated_ffn(attended, w["gate"], w["up"], "silu", gate, up)
        return attended + sg.q4_linear(h, w["down"])

    def _attend(self, q, k, v):
        q, k, v = (t.float().transpose(0, 1).contiguous() for t in (q, k, v))
        s = torch.matmul(q, k.transpose(1, 2).contiguous()) / math.sqrt(q.shape[2])
        s.masked_fill_(torch.ones_like(s[0], dtype=torch.bool).triu(1), float("-inf"))
        return torch.matmul(s.softmax(-1), v).transpose(0, 1).reshape(q.shape[1], -1).to(self.dtype)

    def plain_weight(self, name):
        """A base weight as a 16-bit (or float32) matrix."""
        codes, scales, zeros = self.raw[name]
        k = 2 * codes.shape[1]
        q = torch.stack([codes & 15, codes >> 4], 2).flatten(1).float()
        spread = lambda t: t.float().repeat_interleave(self.group, 1)[:, :k]
        return ((q - spread(zeros)) * spread(scales)).to(self.dtype)


def train_block(layer, x, target, adapter=0, steps=20, lr=3e-4):
    """Fits one adapter of the gated block to ``target`` over a frozen base; returns the losses."""
    Wg, Wu = layer.plain_weight("gate"), layer.plain_weight("up")
    params = [t[adapter].float().clone().requires_grad_() for n in ("gate", "up") for t in layer.lora[n]]
    losses = []
    for _ in range(steps):
        Ag, Bg, Au, Bu = (p.to(layer.dtype) for p in params)
        h = sg.gated_ffn(x, Wg, Wu, "silu", (x @ Ag) @ Bg, (x @ Au) @ Bu)
        loss = (h.float() - target.float()).square().sum(1).mean()
        losses.append(float(loss.detach()))
        grads = torch.autograd.grad(loss, params)
        with torch.no_grad():
            for p, g in zip(params, grads):
                p -= lr * g
    return losses


def main():
    layer = AdaptedLayer(hidden=512, ffn=1376, heads=8, adapters=6, rank=16, dtype=torch.bfloat16)
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(40, 512, generator=gen).bfloat16().cuda()
    row_ids = torch.randint(0, 6, (40,), generator=gen, dtype=torch.int32).sort().values.cuda()
    seg, ids, _ = sg.build_segments(row_ids, 6)
    y = layer.serve(x, torch.arange(40, device="cuda"), (seg, ids))
    print(f"served {tuple(y.shape)}, rms {float(y.float().square().mean().sqrt()):.3f}")
    target = torch.randn(256, 1376, generator=gen).bfloat16().cuda()
    losses = train_block(layer, torch.randn(256, 512, generator=gen).bfloat16().cuda(), target)
    print(f"trained {len(losses)} steps, loss {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
