"""A mixture-of-experts layer with a shared expert: the shared expert trained in 16
bits, then the whole layer served in 4 bits.

    y[t] = Σ_j w[t, j]·expert[id[t, j]](x[t])  +  shared(x[t])

Every step is a call of the library: routing, tables and packing as in 16 bits;
gated_ffn and gated_ffn_backward for the shared expert; mx4_quantize for weights
and activations, mx4_gate_up and mx4_down for the experts (the shared expert is
the same two calls with one expert).

    python examples/moe_layer_4bit.py
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import routed_grouped_gemm_dispatch_gb300 as moe  # noqa: E402


class SharedExpert:
    """The dense gated block with what a training step keeps."""

    def __init__(self, hidden, intermediate, dtype, device, seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def draw(rows, cols):
            return (torch.randn((rows, cols), generator=g, device=device) * cols ** -0.5).to(dtype)

        self.gate_w, self.up_w, self.down_w = draw(intermediate, hidden), draw(intermediate, hidden), draw(hidden, intermediate)
        self.stored = None

    def weights(self):
        return self.gate_w, self.up_w, self.down_w

    def forward(self, x, train=False):
        if not train:
            return moe.gated_ffn(x, *self.weights())
        shape = (x.shape[0], self.gate_w.shape[0])
        s = {k: torch.empty(shape, dtype=x.dtype, device=x.device) for k in ("gate", "up", "up_logits")}
        self.stored = (x, s)
        return moe.gated_ffn(x, *self.weights(), **s)

    def backward(self, d_out):
        """(d_x, d_gate_w, d_up_w, d_down_w) of the last forward(train=True)."""
        x, s = self.stored
        return moe.gated_ffn_backward(d_out, x, *self.weights(), s["gate"], s["up"], s["up_logits"])


def train_shared_expert(expert, teacher, hidden, steps=20, tokens=512, lr=0.2, seed=1234):
    """Plain gradient descent on ‖expert(x) − teacher(x)‖² / 2 per token; the losses."""
    dt, dev = expert.gate_w.dtype, expert.gate_w.device
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    master = [w.float() for w in expert.weights()]
    losses = []
    for _ in range(steps):
        x = torch.randn((tokens, hidden), generator=g, device=dev).to(dt)
        d_out = expert.forward(x, train=True).float() - teacher.forward(x).float()
        losses.append(float(d_out.square().sum()) / (2 * tokens))
        _, *grads = expert.backward(d_out.to(dt))
        for m, d in zip(master, grads):
            m.add_(d.float(), alpha=-lr / tokens)
        expert.gate_w, expert.up_w, expert.down_w = (m.to(dt) for m in master)
    return losses


def route(x, router_w, top_k):
    """Tables, compact weights and every pair's padded row, as the 16-bit layer uses them."""
    ids, weights = moe.router_topk(x, router_w, top_k)
    return tables_of(ids, weights, router_w.shape[0])


def tables_of(ids, weights, experts):
    t = moe.build_dispatch(ids, experts)
    rows = t["group_idx_for_bx"].numel() * moe.BLOCK_TOKEN
    packed = moe.pack_routed(ids, weights, None, t, rows)
    return t, rows, packed["routed_expert_weights"], packed["pair_padded_rows"]


def experts_4bit(x, routing, gate, up, down, out_dtype=torch.float16):
    """Routed experts with 4-bit weights ((codes, scales) stacks); x [T, hidden] 16-bit."""
    t, rows, weights, pair_rows = routing
    tabs = (t["group_sizes"], t["group_offsets"], t["group_padded_offsets"], t["group_idx_for_bx"])
    E, I = gate[0].shape[:2]
    H = x.shape[1]
    # each token is converted once and lands in all its experts' blocks
    xq, xs = moe.mx4_quantize(x, dest_rows=pair_rows, n_dest=rows)
    h = torch.empty((rows, I), dtype=out_dtype, device=x.device)
    moe.mx4_gate_up(xq, xs, *gate, *up, tabs[0], tabs[2], tabs[3], h)
    # only the rows that hold something are converted
    valid = pair_rows.view(-1)
    hq, hs = moe.mx4_quantize(h, src_rows=valid, dest_rows=valid, n_dest=rows)
    out = torch.empty((rows, H), dtype=out_dtype, device=x.device)
    moe.mx4_down(hq, hs, *down, weights, *tabs, out)
    return moe.combine_routed(out, pair_rows)


def experts_16bit(x, ids, weights, gate_w, up_w, down_w):
    t = moe.build_dispatch(ids, gate_w.shape[0])
    rows = t["group_idx_for_bx"].numel() * moe.BLOCK_TOKEN
    p = moe.pack_routed(ids, weights, x, t, rows)
    h = torch.empty((rows, gate_w.shape[1]), dtype=x.dtype, device=x.device)
    out = torch.empty((rows, x.shape[1]), dtype=x.dtype, device=x.device)
    moe.fused_forward(p["stacked_expert_tokens"], gate_w, up_w, down_w, p["routed_expert_weights"], t["group_sizes"],
                      t["group_offsets"], t["group_padded_offsets"], t["group_idx_for_bx"], h, out)
    return moe.combine_routed(out, p["pair_padded_rows"])


class Layer:
    def __init__(self, hidden=2048, intermediate=1408, experts=64, top_k=6, shared=2816, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def draw(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5).half()

        self.top_k, self.device = top_k, device
        self.router_w = draw(experts, hidden)
        self.gate_w, self.up_w = draw(experts, intermediate, hidden), draw(experts, intermediate, hidden)
        self.down_w = draw(experts, hidden, intermediate)
        self.shared = SharedExpert(hidden, shared, torch.float16, device, seed + 1)
        self.q = None

    def forward_16bit(self, x):
        ids, w = moe.router_topk(x, self.router_w, self.top_k)
        return experts_16bit(x, ids, w, self.gate_w, self.up_w, self.down_w) + self.shared.forward(x)

    def quantize(self):
        """4-bit weights, laid out once."""
        s = self.shared
        self.q = {"routed": [moe.mx4_quantize(w) for w in (self.gate_w, self.up_w, self.down_w)],
                  "shared": [moe.mx4_quantize(w[None]) for w in s.weights()]}

    def forward_4bit(self, x):
        T = x.shape[0]
        everyone = tables_of(torch.zeros((T, 1), dtype=torch.int32, device=x.device),
                             torch.ones((T, 1), dtype=torch.float32, device=x.device), 1)
        return (experts_4bit(x, route(x, self.router_w, self.top_k), *self.q["routed"])
                + experts_4bit(x, everyone, *self.q["shared"]))


def milliseconds(fn, reps=20):
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(reps):
        fn()
    torch.cuda.synchronize()
    return (time.perf_counter() - t0) / reps * 1e3


def main():
    torch.manual_seed(0)
    layer = Layer()
    hidden = layer.router_w.shape[1]
    teacher = SharedExpert(hidden, layer.shared.gate_w.shape[0], torch.float16, layer.device, seed=9)
    losses = train_shared_expert(layer.shared, teacher, hidden)
    print(f"shared expert: loss {losses[0]:.1f} -> {losses[-1]:.1f} in {len(losses)} steps")
    layer.quantize()
    for tokens in (1, 64, 4096):
        x = torch.randn((tokens, hidden), device=layer.device).half()
        y16, y4 = layer.forward_16bit(x).float(), layer.forward_4bit(x).float()
        print(f"{tokens:5d} tokens: 4-bit against 16-bit, relative difference {float((y4 - y16).norm() / y16.norm()):.3f}; "
              f"{milliseconds(lambda: layer.forward_16bit(x)):.3f} ms in 16 bits, "
              f"{milliseconds(lambda: layer.forward_4bit(x)):.3f} ms in 4 bits")


if __name__ == "__main__":
    main()
