"""Cases of the operators that train a routed layer: the router's balance and z losses with
its per-expert counts, the router's gradients, and the orthogonalised update of weight
matrices; each in a plain form of elementary torch operations and as calls of the library.

Operators:
  balance    from the router's logits z [T, E] and chosen experts [T, k], over the valid tokens
             (T of them in all, T_s in sequence s) with p = softmax(z):
               counts[s, e]  pairs of sequence s that chose expert e
               balance = E / (k T) · Σ_s 1/T_s · Σ_e counts[s, e] · Σ_t∈s p[t, e]
               z_loss  = 1/T · Σ_t logsumexp(z[t])²
  backward   gradients of the tokens and of the router's weights from those of the routed
             weights w[t, j] = p[t, id[t, j]] and of the two losses (counts are constants):
               g[t, e] = d_balance · E / (k T T_s) · counts[s, e] + Σ_j [id[t, j] = e] · d_w[t, j]
               d_z = p ⊙ (g − Σ_e p g) + d_z_loss · 2/T · logsumexp(z) · p
               d_x = d_z·W,  d_W = d_zᵀ·x;  a token that is not valid has d_z = 0
  ortho      X₀ = G / max(‖G‖, eps) (Frobenius), then five times
               A = X·Xᵀ,  X ← a·X + (b·A + c·A²)·X
             of fp16, bf16 or fp32 matrices (a stack of them), in bf16
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
BIG_TOKENS, BIG_EXPERTS, BIG_HIDDEN = 16384, 256, 7168
BIG_STACK = (64, 1408, 2048)


def listed():
    return [
        # a decode-sized batch of a fine-tuning step: one short sequence
        {"name": "balance 32x128", "op": "balance", "tokens": 32, "experts": 128, "top_k": 8, "seqs": 1,
         "masked": False},
        # DeepSeek-V2-Lite-shaped routing of five packed sequences of unequal lengths, some padding in them
        {"name": "balance 4097x64", "op": "balance", "tokens": 4097, "experts": 64, "top_k": 6, "seqs": 5,
         "masked": True},
        # a DeepSeek-V3-shaped training batch, four packed sequences
        {"name": "balance 16384x256", "op": "balance", "tokens": 16384, "experts": 256, "top_k": 8, "seqs": 4,
         "masked": False},
        # the router's gradients for the same three
        {"name": "router grad 32x128", "op": "backward", "tokens": 32, "experts": 128, "top_k": 8, "seqs": 1,
         "masked": False, "hidden": 2048, "dtype": "fp16"},
        {"name": "router grad 4097x64", "op": "backward", "tokens": 4097, "experts": 64, "top_k": 6, "seqs": 5,
         "masked": True, "hidden": 2048, "dtype": "bf16"},
        {"name": "router grad 16384x256", "op": "backward", "tokens": 16384, "experts": 256, "top_k": 8, "seqs": 4,
         "masked": False, "hidden": 7168, "dtype": "fp16"},
        # the update of the DeepSeek-V2-Lite-shaped router's own weights
        {"name": "ortho router", "op": "ortho", "batch": 1, "rows": 64, "cols": 2048, "dtype": "bf16"},
        # a few small matrices of no round size, as adapters have
        {"name": "ortho odd stack", "op": "ortho", "batch": 3, "rows": 333, "cols": 1001, "dtype": "fp16"},
        # a shared expert's gate weights, more rows than columns
        {"name": "ortho shared gate", "op": "ortho", "batch": 1, "rows": 2816, "cols": 2048, "dtype": "bf16"},
        # a DeepSeek-V3-shaped shared expert's last weights, momentum kept in 32 bits
        {"name": "ortho dsv3 down", "op": "ortho", "batch": 1, "rows": 7168, "cols": 2048, "dtype": "fp32"},
        # all routed experts' gate weights of a DeepSeek-V2-Lite-shaped layer
        {"name": "ortho experts", "op": "ortho", "batch": 64, "rows": 1408, "cols": 2048, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step):
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["balance", "backward", "backward", "ortho", "ortho", "ortho"])
    if op == "ortho":
        big = work({"op": op, "batch": BIG_STACK[0], "rows": BIG_STACK[1], "cols": BIG_STACK[2], "dtype": "bf16"})
        while True:
            step = rng.choice([1, 8, 128])
            c = {"op": op, "batch": rng.choice([1, 1, 2, 5, 16, 64]), "rows": _size(rng, 16, 7168, step),
                 "cols": _size(rng, 16, 7168, step), "dtype": rng.choice(["fp16", "bf16", "fp32"])}
            w = work(c)
            if w["flops"] <= big["flops"] and w["bytes"] <= big["bytes"]:
                return c
    experts = _log(rng, 4, BIG_EXPERTS)
    tokens = _log(rng, 1, BIG_TOKENS)
    c = {"op": op, "tokens": tokens, "experts": experts, "top_k": rng.randint(1, min(8, experts)),
         "seqs": rng.choice([1, 1, 2, 7]), "masked": rng.random() < 0.5}
    if op == "backward":
        c["hidden"], c["dtype"] = _size(rng, 128, BIG_HIDDEN, rng.choice([8, 128])), rng.choice(["fp16", "bf16"])
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _routing(case, g):
    """Logits whose experts are unequally popular, the chosen experts, sequences and mask."""
    T, E = case["tokens"], case["experts"]
    z = torch.randn((T, E), generator=g, device=DEV)
    z -= 0.5 * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    s = {"logits": z, "ids": torch.topk(z, case["top_k"], dim=1).indices.to(torch.int32), "offsets": None,
         "mask": None}
    if case["seqs"] > 1:
        cuts = torch.randint(0, T + 1, (case["seqs"] - 1,), generator=g, device=DEV).sort().values
        ends = torch.tensor([0, T], device=DEV)
        s["offsets"] = torch.cat((ends[:1], cuts, ends[1:])).to(torch.int32)
    if case["masked"]:
        s["mask"] = torch.rand((T,), generator=g, device=DEV) >= 0.05
    return s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "ortho":
        # a momentum: a few strong directions over noise, of a gradient's size
        B, m, n = case["batch"], case["rows"], case["cols"]
        r = max(1, min(m, n) // 16)
        u = torch.randn((B, m, r), generator=g, device=DEV).mul_(1e-3 * r ** -0.5)
        x = torch.bmm(u, torch.randn((B, r, n), generator=g, device=DEV))
        x += torch.randn((B, m, n), generator=g, device=DEV).mul_(3e-4)
        return {"case": case, "update": x.to(DT[case["dtype"]])}
    s = {"case": case, **_routing(case, g)}
    if case["op"] == "balance":
        return s
    T, E, H, dt = case["tokens"], case["experts"], case["hidden"], DT[case["dtype"]]
    s["x"] = torch.randn((T, H), generator=g, device=DEV).to(dt)
    s["w"] = torch.randn((E, H), generator=g, device=DEV).mul_(H ** -0.5).to(dt)
    # gradients of a mean over tokens, times a loss scale that leaves none above 64
    scale = min(4096.0, 64.0 * T)
    s["d_weights"] = torch.randn((T, case["top_k"]), generator=g, device=DEV).mul_(scale / T)
    s["d_losses"] = torch.tensor([0.01 * scale, 0.001 * scale], device=DEV)
    valid, seq = _sequences(s)
    s["counts"], s["seq_tokens"] = _counts(s, valid, seq)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _sequences(s):
    """Of each token: is it valid, and which sequence is it in."""
    T = s["logits"].shape[0]
    t = torch.arange(T, device=DEV)
    seq = torch.zeros_like(t) if s["offsets"] is None else torch.searchsorted(s["offsets"][1:-1].contiguous(), t,
                                                                               right=True, out_int32=False)
    valid = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"]
    return valid, seq


def _counts(s, valid, seq):
    S, E = s["case"]["seqs"], s["case"]["experts"]
    k = s["ids"].shape[1]
    one = valid.to(torch.int32)
    counts = torch.zeros(S * E, dtype=torch.int32, device=DEV)
    counts.index_add_(0, (seq[:, None] * E + s["ids"]).reshape(-1), one[:, None].expand(-1, k).reshape(-1))
    tokens = torch.zeros(S, dtype=torch.int32, device=DEV).index_add_(0, seq, one)
    return counts.view(S, E), torch.cat((tokens, tokens.sum().to(torch.int32)[None]))


def _run_own(s):
    import routed_grouped_gemm_dispatch_gb300 as moe
    case = s["case"]
    if case["op"] == "ortho":
        return moe.orthogonalize(s["update"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
    if case["op"] == "balance":
        return moe.router_balance(s["logits"], s["ids"], token_mask=s["mask"], seq_offsets=s["offsets"])
    return moe.router_backward(s["x"], s["w"], s["logits"], s["ids"], d_topk_weights=s["d_weights"],
                               d_losses=s["d_losses"], counts=s["counts"], seq_tokens=s["seq_tokens"],
                               token_mask=s["mask"], seq_offsets=s["offsets"])


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    if case["op"] == "ortho":
        a, b, c = COEFFICIENTS
        x = s["update"].float()
        # the norm of many small squares: summed in 64 bits
        norm = x.double().square_().sum(dim=(1, 2), keepdim=True).sqrt_().clamp_(min=EPS)
        x = x / norm.float()
        tall = case["rows"] > case["cols"]
        if tall:
            x = x.transpose(1, 2).contiguous()
        for _ in range(STEPS):
            gram = torch.bmm(x, x.transpose(1, 2))
            x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
        return (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()
    E, k = case["experts"], case["top_k"]
    valid, seq = _sequences(s)
    z = s["logits"]
    top = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(dim=1, keepdim=True)
    p = e / total
    lse = top[:, 0] + torch.log(total[:, 0])
    if case["op"] == "balance":
        counts, tokens = _counts(s, valid, seq)
        v = valid.double()
        per_seq = torch.zeros((case["seqs"], E), dtype=torch.float64, device=DEV)
        per_seq.index_add_(0, seq, p.double() * v[:, None])
        n = tokens[-1].double().clamp(min=1)
        balance = ((counts.double() * per_seq).sum(dim=1) / tokens[:-1].double().clamp(min=1)).sum() * E / (k * n)
        z_loss = (lse.double().square() * v).sum() / n
        return torch.stack((balance, z_loss)).float(), counts, tokens
    n = s["seq_tokens"].float().clamp(min=1)
    d_bal, d_zl = s["d_losses"][0], s["d_losses"][1]
    share = d_bal * E / (k * n[-1]) * s["counts"].float() / n[:-1, None]
    g = share[seq]
    g.scatter_add_(1, s["ids"].long(), s["d_weights"])
    d_z = p * (g - (p * g).sum(dim=1, keepdim=True)) + d_zl * (2 / n[-1]) * lse[:, None] * p
    d_z = d_z * valid[:, None]
    return (d_z @ s["w"].float()).to(s["x"].dtype), (d_z.t() @ s["x"].float()).to(s["x"].dtype)


# ---------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "ortho" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "ortho":
        a, b, c = COEFFICIENTS
        out = torch.empty(s["update"].shape, dtype=torch.float64, device=DEV)
        for i, g in enumerate(s["update"]):
            x = g.double()
            x = x / max(float(torch.linalg.vector_norm(x)), EPS)
            for _ in range(STEPS):
                # on the shorter side; the same polynomial from either side
                if x.shape[0] <= x.shape[1]:
                    gram = torch.einsum("ik,jk->ij", x, x)
                    x = a * x + torch.einsum("ij,jk->ik", gram, torch.einsum("ij,jk->ik", b * torch.eye(
                        len(gram), dtype=x.dtype, device=DEV) + c * gram, x))
                else:
                    gram = torch.einsum("ki,kj->ij", x, x)
                    x = a * x + torch.einsum("ki,ij->kj", torch.einsum("ki,ij->kj", x, b * torch.eye(
                        len(gram), dtype=x.dtype, device=DEV) + c * gram), gram)
            out[i] = x
        return out
    T, E, k, S = case["tokens"], case["experts"], case["top_k"], case["seqs"]
    z = s["logits"].double()
    p = torch.softmax(z, dim=1)
    lse = torch.logsumexp(z, dim=1)
    bounds = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    ok = [True] * T if s["mask"] is None else s["mask"].tolist()
    rows = [[t for t in range(lo, hi) if ok[t]] for lo, hi in zip(bounds, bounds[1:])]
    rows = [torch.tensor(r, dtype=torch.int64, device=DEV) for r in rows]
    total = sum(len(r) for r in rows)
    chosen = torch.zeros((T, E), dtype=torch.float64, device=DEV)
    for j in range(k):
        chosen[torch.arange(T, device=DEV), s["ids"][:, j].long()] += 1
    counts = [chosen[r].sum(dim=0) for r in rows]
    if case["op"] == "balance":
        balance = sum(float((c * p[r].sum(dim=0)).sum()) / len(r) for c, r in zip(counts, rows) if len(r))
        z_loss = sum(float((lse[r] ** 2).sum()) for r in rows)
        losses = torch.tensor([balance * E / (k * max(total, 1)), z_loss / max(total, 1)], dtype=torch.float64)
        return losses, torch.stack(counts), torch.tensor([len(r) for r in rows] + [total], dtype=torch.float64)
    # the gradients by the chain rule, from the loss itself
    z = z.requires_grad_()
    x, w = s["x"].double(), s["w"].double()
    with torch.enable_grad():
        p = torch.softmax(z, dim=1)
        sq = torch.logsumexp(z, dim=1) ** 2
        loss = z.new_zeros(())
        for c, r in zip(counts, rows):
            if len(r):
                loss = loss + float(s["d_losses"][0].double()) * E / (k * total * len(r)) * (c * p[r].sum(dim=0)).sum()
                loss = loss + float(s["d_losses"][1].double()) / total * sq[r].sum()
                loss = loss + (p[r].gather(1, s["ids"][r].long()) * s["d_weights"][r].double()).sum()
    d_z, = torch.autograd.grad(loss, z) if total else (torch.zeros_like(z),)
    return torch.einsum("te,eh->th", d_z, w), torch.einsum("te,th->eh", d_z, x)


def work(case):
    b = {"fp16": 2, "bf16": 2, "fp32": 4}
    if case["op"] == "ortho":
        B, m, n = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        # X·Xᵀ and A² are symmetric: half of their products
        return {"bytes": B * m * n * (b[case["dtype"]] + 2), "flops": STEPS * B * (3 * m * m * n + m ** 3)}
    T, E, k, S = case["tokens"], case["experts"], case["top_k"], case["seqs"]
    routing = 4 * T * E + 4 * T * k + 4 * S * E + (T if case["masked"] else 0)
    if case["op"] == "balance":
        return {"bytes": routing, "flops": 5 * T * E}
    H = case["hidden"]
    return {"bytes": routing + 4 * T * k + 2 * (2 * T * H + 2 * E * H), "flops": 4 * T * E * H}
