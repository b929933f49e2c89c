"""A mixture-of-experts layer with a shared expert: the shared expert trained in 16
bits, the router trained to spread its tokens over the experts, then the whole layer served in 4 bits.

    y[t] = Σ_j w[t, j]·expert[id[t, j]](x[t])  +  shared(x[t])

Every step is a call of the library: routing, tables and packing as in 16 bits;
gated_ffn and gated_ffn_backward for the shared expert, router_balance and router_backward
for the router, orthogonalize for both's updates; mx4_quantize for weights
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


def orthogonal_step(master, grad, lr):
    """master −= lr · √max(1, rows/cols) · orthogonalised grad: an update whose singular values are alike."""
    master.add_(moe.orthogonalize(grad).float(), alpha=-lr * max(1.0, master.shape[-2] / master.shape[-1]) ** 0.5)


def train_shared_expert(expert, teacher, hidden, steps=20, tokens=512, lr=0.2, seed=1234, orthogonal=False):
    """Gradient descent on ‖expert(x) − teacher(x)‖² / 2 per token, plain or with orthogonalised updates; the losses."""
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
            if orthogonal:
                orthogonal_step(m, d, lr)
            else:
                m.add_(d.float(), alpha=-lr / tokens)
        expert.gate_w, expert.up_w, expert.down_w = (m.to(dt) for m in master)
    return losses


def balance_step(x, router_w, top_k, balance_weight=1.0, z_weight=1e-3, scale=1024.0, **sequences):
    """The router's losses, its counts per sequence and expert, and the gradient of its weights from
    balance_weight · balance loss + z_weight · z loss.  ``scale``: of the gradients while they are
    16-bit; ``sequences``: token_mask and seq_offsets where x holds packed or padded sequences."""
    logits = torch.empty((x.shape[0], router_w.shape[0]), dtype=torch.float32, device=x.device)
    ids, _ = moe.router_topk(x, router_w, top_k, logits=logits)
    losses, counts, tokens = moe.router_balance(logits, ids, **sequences)
    d_losses = torch.tensor([balance_weight * scale, z_weight * scale], device=x.device)
    _, d_w = moe.router_backward(x, router_w, logits, ids, d_losses=d_losses, counts=counts, seq_tokens=tokens, **sequences)
    return losses, counts, d_w.float() / scale


def train_router(layer, x, steps=20, lr=0.02):
    """Spreads the tokens of x over the layer's experts; (balance loss, z loss) of every step."""
    master, seen = layer.router_w.float(), []
    for _ in range(steps):
        losses, _, d_w = balance_step(x, layer.router_w, layer.top_k)
        seen.append(losses)
        orthogonal_step(master, d_w, lr)
        layer.router_w = master.half()
    return torch.stack(seen).tolist()


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
    x = torch.randn((4096, hidden), device=layer.device).half() + 0.1 * layer.router_w[:4].sum(0)
    losses = train_router(layer, x)
    print(f"router: balance loss {losses[0][0]:.3f} -> {losses[-1][0]:.3f} in {len(losses)} steps (1 is even)")
    layer.quantize()
    for tokens in (1, 64, 4096):
        x = torch.randn((tokens, hidden), device=layer.device).half()
        y16, y4 = layer.forward_16bit(x).float(), layer.forward_4bit(x).float()
        print(f"{tokens:5d} tokens: 4-bit against 16-bit, relative difference {float((y4 - y16).norm() / y16.norm()):.3f}; "
              f"{milliseconds(lambda: layer.forward_16bit(x)):.3f} ms in 16 bits, "
              f"{milliseconds(lambda: layer.forward_4bit(x)):.3f} ms in 4 bits")


if __name__ == "__main__":
    main()
