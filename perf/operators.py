"""Cases of the dense gated feed-forward block (forward and gradients) and of the
4-bit microscaled operators (quantisation, grouped and dense products), each in a
plain form of elementary torch operations and as calls of the library.

Operators:
  ffn           y = (silu(x·gate_wᵀ) ⊙ (x·up_wᵀ))·down_wᵀ; the training form also
                returns the gate and up values and their gated product
  ffn_backward  gradients of x and of the three weights from d_y and the stored
                gate, up and gated values
  mx4_quantize  microscaled 4-bit codes (e2m1, blocks of 32, a power-of-two scale)
                and back to the values they stand for
  mx4_product   products of 4-bit operands: "gate_up" and "down" over rows grouped by
                expert in padded 128-row blocks, "matmul" over plain rows
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BT = 128                      # rows of a block of the grouped layout
BLOCK = 32                    # values that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BIG_FLOPS = 12 * 8192 * 7168 * 2048          # the largest listed case
BIG_QUANT = 16384 * 7168


def listed():
    return [
        # one token through a DeepSeek-V3-shaped shared expert: a single stream's decode step
        {"name": "ffn 1 token", "op": "ffn", "tokens": 1, "hidden": 7168, "inter": 2048, "dtype": "bf16",
         "train": False},
        # a small decode batch through DeepSeek-V2-Lite-shaped shared experts (two of 1408)
        {"name": "ffn 37 tokens", "op": "ffn", "tokens": 37, "hidden": 2048, "inter": 2816, "dtype": "fp16",
         "train": False},
        # a prompt whose length is no multiple of anything, forward of a training step
        {"name": "ffn train 4097", "op": "ffn", "tokens": 4097, "hidden": 2048, "inter": 2816, "dtype": "bf16",
         "train": True},
        # a long prefill batch through the DeepSeek-V3-shaped shared expert
        {"name": "ffn 8192", "op": "ffn", "tokens": 8192, "hidden": 7168, "inter": 2048, "dtype": "bf16",
         "train": False},
        # a short ragged micro-batch's gradients
        {"name": "ffn backward 301", "op": "ffn_backward", "tokens": 301, "hidden": 2048, "inter": 2816,
         "dtype": "fp16"},
        # a training batch's gradients at the DeepSeek-V3 shape
        {"name": "ffn backward 8192", "op": "ffn_backward", "tokens": 8192, "hidden": 7168, "inter": 2048,
         "dtype": "bf16"},
        # a decode batch's activations to 4 bits
        {"name": "mx4 quantize 33", "op": "mx4_quantize", "rows": 33, "cols": 2048, "dtype": "fp16"},
        # a DeepSeek-V3-shaped prefill batch's activations (and the size of a few experts' weights)
        {"name": "mx4 quantize 16384", "op": "mx4_quantize", "rows": 16384, "cols": 7168, "dtype": "bf16"},
        # decode, 32 tokens with skewed experts: most weight bytes are read for one or two rows
        {"name": "mx4 gate_up decode", "op": "mx4_product", "form": "gate_up", "tokens": 32, "top_k": 8,
         "experts": 128, "k": 2048, "n": 768, "zipf": 1.2, "dtype": "fp16"},
        # DeepSeek-V2-Lite-shaped prefill, first half of the routed experts
        {"name": "mx4 gate_up dsv2_lite", "op": "mx4_product", "form": "gate_up", "tokens": 4096, "top_k": 6,
         "experts": 64, "k": 2048, "n": 1408, "zipf": 0.0, "dtype": "fp16"},
        # a slice of the DeepSeek-V3-shaped prefill, second half of the routed experts
        {"name": "mx4 down dsv3_slice", "op": "mx4_product", "form": "down", "tokens": 2048, "top_k": 8,
         "experts": 32, "k": 2048, "n": 7168, "zipf": 1.0, "dtype": "fp16"},
        # the shared expert's last product in 4 bits, an odd number of tokens
        {"name": "mx4 matmul 1111", "op": "mx4_product", "form": "matmul", "tokens": 1111, "top_k": 1,
         "experts": 1, "k": 2048, "n": 7168, "zipf": 0.0, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step):
    n = max(lo, _log(rng, lo, hi) // step * step)
    return n + step if n == 3072 else n


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_backward", "mx4_quantize", "mx4_product", "mx4_product"])
    if op in ("ffn", "ffn_backward"):
        while True:
            c = {"op": op, "tokens": _size(rng, 1, 8192, 1), "hidden": _size(rng, 512, 7168, rng.choice([8, 128])),
                 "inter": _size(rng, 512, 4096, rng.choice([8, 128])), "dtype": rng.choice(["fp16", "bf16"])}
            if op == "ffn":
                c["train"] = rng.random() < 0.4
            if work(c)["flops"] <= BIG_FLOPS:
                return c
    if op == "mx4_quantize":
        while True:
            c = {"op": op, "rows": _size(rng, 1, 16384, 1), "cols": _size(rng, 128, 14336, 128),
                 "dtype": rng.choice(["fp16", "bf16", "fp32"])}
            if c["rows"] * c["cols"] <= BIG_QUANT:
                return c
    while True:
        form = rng.choice(["gate_up", "down", "matmul"])
        experts = 1 if form == "matmul" else rng.choice([4, 8, 32, 64, 128])
        c = {"op": op, "form": form, "tokens": _size(rng, 1, 4096, 1), "top_k": 1 if experts == 1 else rng.choice([2, 4]),
             "experts": experts, "k": _size(rng, 256, 7168, 128), "n": _size(rng, 256, 7168, 128),
             "zipf": 0.0 if experts == 1 else rng.choice([0.0, 1.0, 1.2]), "dtype": rng.choice(["fp16", "bf16"])}
        if work(c)["flops"] <= BIG_FLOPS // 4 and experts * c["k"] * c["n"] <= 32 * 7168 * 2048:
            return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dtype)


def _pow2(e):
    """2^e in fp32 from whole numbers e in [-127, 127], by its bits (2^-127 is subnormal)."""
    e = e.to(torch.int32)
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _quant(x):
    """Codes 0..15 [rows, cols] and scale bytes [rows, cols / 32] of fp32 values."""
    rows, cols = x.shape
    b = x.view(rows, cols // BLOCK, BLOCK)
    a = b.abs().amax(2)
    e = (torch.frexp(a)[1] - 3).clamp(-127, 127)          # frexp: a = m * 2^n with m in [0.5, 1)
    e = torch.where(a == 0, torch.full_like(e, -127), e)
    v = (b * _pow2(-e)[..., None]).abs()
    # halfway points between neighbouring values; a tie goes to the even code
    c = ((v > 0.25).byte() + (v >= 0.75).byte() + (v > 1.25).byte() + (v >= 1.75).byte()
         + (v > 2.5).byte() + (v >= 3.5).byte() + (v > 5.0).byte())
    c = c | (torch.signbit(b).byte() << 3)
    return c.view(rows, cols), (e + 127).to(torch.uint8)


def _pack(codes):
    """Two codes to a byte, the even column in the low half."""
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _tiles(scales):
    """Scale bytes [rows, blocks] in tiles of 128 rows x 4 blocks:
    [row // 128, block // 4, row % 32, row // 32 % 4, block % 4]."""
    rows, blocks = scales.shape
    r = -(-rows // 128)
    t = torch.zeros((r * 128, blocks), dtype=torch.uint8, device=scales.device)
    t[:rows] = scales
    return t.view(r, 4, 32, blocks // 4, 4).permute(0, 3, 2, 1, 4).contiguous()


def _untile(t):
    r, kb = t.shape[:2]
    return t.permute(0, 3, 2, 1, 4).reshape(r * 128, kb * 4)


def _unpack(packed, tiles):
    """fp32 values [rows, cols] of packed codes and tiled scales."""
    rows, half = packed.shape
    c = torch.stack((packed & 15, packed >> 4), dim=2).view(rows, 2 * half).to(torch.int32)
    v = torch.tensor(E2M1, device=packed.device)[c & 7] * (1 - 2 * (c >> 3))
    s = _pow2(_untile(tiles)[:rows].to(torch.int32) - 127)
    return (v.view(rows, -1, BLOCK) * s[..., None]).view(rows, 2 * half)


def _routing(case, g):
    """Distinct experts of each token; None of them is chosen twice by a token."""
    E = case["experts"]
    p = -case["zipf"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    u = torch.rand((case["tokens"], E), generator=g, device=DEV).clamp_(1e-9, 1 - 1e-7)
    return torch.topk(p - torch.log(-torch.log(u)), case["top_k"], dim=1).indices


def _mx4_random(g, rows, cols, std):
    """4-bit operand of normal values, made in pieces of at most 64 Mi values."""
    step = max(128, (64 << 20) // cols // 128 * 128)
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=DEV)
    tiles = torch.empty((-(-rows // 128), cols // 128, 32, 4, 4), dtype=torch.uint8, device=DEV)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        c, s = _quant(torch.randn((n, cols), generator=g, device=DEV).mul_(std))
        codes[r:r + n] = _pack(c)
        tiles[r // 128:(r + n + 127) // 128] = _tiles(s)
    return codes, tiles


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "mx4_quantize":
        # activations: normal with a few loud channels, as a norm's output has
        x = torch.randn((case["rows"], case["cols"]), generator=g, device=DEV)
        x *= torch.exp(torch.randn((1, case["cols"]), generator=g, device=DEV))
        return {"case": case, "x": x.to(DT[case["dtype"]])}
    if op in ("ffn", "ffn_backward"):
        dt, T, H, I = DT[case["dtype"]], case["tokens"], case["hidden"], case["inter"]
        s = {"case": case, "x": _normal(g, (T, H), 1.0, dt), "gate_w": _normal(g, (I, H), H ** -0.5, dt),
             "up_w": _normal(g, (I, H), H ** -0.5, dt), "down_w": _normal(g, (H, I), I ** -0.5, dt)}
        if op == "ffn_backward":
            s["d_y"] = _normal(g, (T, H), 1.0, dt)
            # what the forward stored
            gate, up = s["x"].float() @ s["gate_w"].float().t(), s["x"].float() @ s["up_w"].float().t()
            s["gate"], s["up"], s["h"] = gate.to(dt), up.to(dt), (gate * torch.sigmoid(gate) * up).to(dt)
        return s
    # mx4_product
    dt, K, N, E = DT[case["dtype"]], case["k"], case["n"], case["experts"]
    s = {"case": case}
    if case["form"] == "matmul":
        rows = case["tokens"]
        s["a"], s["a_scales"] = _mx4_random(g, rows, K, 1.0)
        s["b"], s["b_scales"] = _mx4_random(g, N, K, K ** -0.5)
        s["out"] = torch.zeros((rows, N), dtype=dt, device=DEV)
        return s
    ids = _routing(case, g)
    sizes = torch.bincount(ids.reshape(-1), minlength=E)
    padded = (sizes + 1 + BT - 1) // BT * BT
    starts = torch.cumsum(padded, 0) - padded
    offsets = torch.cumsum(sizes, 0) - sizes
    blocks = -(-ids.numel() // BT) + E
    first = torch.arange(blocks, device=DEV) * BT
    s["sizes"], s["offsets"], s["padded"] = (t.to(torch.int32) for t in (sizes, offsets, starts))
    s["gidx"] = (torch.searchsorted(starts, first, right=True) - 1).to(torch.int32)
    rows = blocks * BT
    s["a"], s["a_scales"] = _mx4_random(g, rows, K, 1.0)
    n_rows = 2 * N if case["form"] == "gate_up" else N
    b, b_scales = _mx4_random(g, E * n_rows, K, K ** -0.5)
    if case["form"] == "gate_up":
        s["b"], s["b2"] = b[:E * N].view(E, N, K // 2), b[E * N:].view(E, N, K // 2)
        s["b_scales"], s["b2_scales"] = b_scales[:E * N // 128], b_scales[E * N // 128:]
    else:
        s["b"], s["b_scales"] = b.view(E, N, K // 2), b_scales
        s["weights"] = torch.rand((ids.numel(),), generator=g, device=DEV)
    s["out"] = torch.zeros((rows, N), dtype=dt, device=DEV)
    # each expert's rows side by side, for the plain form: [E, most rows of an expert]
    most = int(sizes.max())
    m = torch.arange(most, device=DEV)
    s["grid"] = (starts[:, None] + m).clamp_(max=rows - 1)
    s["slot"] = torch.nonzero((m < sizes[:, None]).reshape(-1)).view(-1)
    s["valid"] = s["grid"].reshape(-1)[s["slot"]]
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _run_own(s):
    import routed_grouped_gemm_dispatch_gb300 as moe
    case, op = s["case"], s["case"]["op"]
    if op == "ffn":
        if not case["train"]:
            return {"y": moe.gated_ffn(s["x"], s["gate_w"], s["up_w"], s["down_w"])}
        gate = torch.empty((case["tokens"], case["inter"]), dtype=s["x"].dtype, device=s["x"].device)
        up, h = torch.empty_like(gate), torch.empty_like(gate)
        y = moe.gated_ffn(s["x"], s["gate_w"], s["up_w"], s["down_w"], up_logits=h, gate=gate, up=up)
        return {"y": y, "gate": gate, "up": up, "h": h}
    if op == "ffn_backward":
        return moe.gated_ffn_backward(s["d_y"], s["x"], s["gate_w"], s["up_w"], s["down_w"], s["gate"], s["up"],
                                      s["h"])
    if op == "mx4_quantize":
        codes, scales = moe.mx4_quantize(s["x"])
        return moe.mx4_dequantize(codes, scales, s["x"].dtype)
    if case["form"] == "matmul":
        return moe.mx4_matmul(s["a"], s["a_scales"], s["b"], s["b_scales"], s["out"])
    if case["form"] == "gate_up":
        return moe.mx4_gate_up(s["a"], s["a_scales"], s["b"], s["b_scales"], s["b2"], s["b2_scales"], s["sizes"],
                               s["padded"], s["gidx"], s["out"])
    return moe.mx4_down(s["a"], s["a_scales"], s["b"], s["b_scales"], s["weights"], s["sizes"], s["offsets"],
                        s["padded"], s["gidx"], s["out"])


def run(s):
    if own:
        return _run_own(s)
    case, op = s["case"], s["case"]["op"]
    if op == "mx4_quantize":
        c, sc = _quant(s["x"].float())
        return _unpack(_pack(c), _tiles(sc)).to(s["x"].dtype)
    if op == "ffn":
        dt = s["x"].dtype
        x = s["x"].float()
        gate, up = x @ s["gate_w"].float().t(), x @ s["up_w"].float().t()
        h = gate / (1 + torch.exp(-gate)) * up
        y = (h @ s["down_w"].float().t()).to(dt)
        return {"y": y, "gate": gate.to(dt), "up": up.to(dt), "h": h.to(dt)} if case["train"] else {"y": y}
    if op == "ffn_backward":
        dt = s["x"].dtype
        gate, up, d_y, x = s["gate"].float(), s["up"].float(), s["d_y"].float(), s["x"].float()
        sig = 1 / (1 + torch.exp(-gate))
        d_h = d_y @ s["down_w"].float()
        d_gate, d_up = d_h * up * sig * (1 + gate * (1 - sig)), d_h * gate * sig
        d_x = d_gate @ s["gate_w"].float() + d_up @ s["up_w"].float()
        return (d_x.to(dt), (d_gate.t() @ x).to(dt), (d_up.t() @ x).to(dt), (d_y.t() @ s["h"].float()).to(dt))
    out = s["out"]
    a = _unpack(s["a"], s["a_scales"])
    if case["form"] == "matmul":
        return out.copy_((a @ _unpack(s["b"], s["b_scales"]).t()).to(out.dtype))
    E, N, half = s["b"].shape
    a = a[s["grid"]]                                                   # [E, most, K]
    c = torch.bmm(a, _unpack(s["b"].view(E * N, half), s["b_scales"]).view(E, N, 2 * half).transpose(1, 2))
    if case["form"] == "gate_up":
        up = torch.bmm(a, _unpack(s["b2"].view(E * N, half), s["b2_scales"]).view(E, N, 2 * half).transpose(1, 2))
        c = c / (1 + torch.exp(-c)) * up
        c = c.view(-1, N)[s["slot"]]
    else:
        c = c.view(-1, N)[s["slot"]] * s["weights"][:, None]          # slots run in compact order
    out[s["valid"]] = c.to(out.dtype)
    return out


# ---------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------

def _two_to(e):
    """2^e in fp64 from whole numbers e, by its exponent bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(packed, tiles):
    """fp64 values, from each code's sign, exponent and fraction bits."""
    rows = packed.shape[0]
    c = torch.empty((rows, 2 * packed.shape[1]), dtype=torch.int16, device=packed.device)
    c[:, 0::2], c[:, 1::2] = (packed % 16).to(torch.int16), (packed // 16).to(torch.int16)
    sign, ex, frac = c // 8, c % 8 // 2, c % 2
    v = torch.where(ex == 0, frac.double() * 0.5, (1 + 0.5 * frac.double()) * _two_to(ex - 1))
    v = torch.where(sign == 1, -v, v)
    r, b = torch.arange(rows, device=packed.device), torch.arange(c.shape[1], device=packed.device) // BLOCK
    sc = tiles[(r // 128)[:, None], b // 4, (r % 32)[:, None], (r // 32 % 4)[:, None], b % 4]
    return v * _two_to(sc.to(torch.int64) - 127)


def _exact_quant(x):
    """Round trip in 64 bits: the nearest representable value by distance, of two the one with the even code."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    mags = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    step = max(1, (4 << 20) // x.shape[1])
    for r in range(0, x.shape[0], step):
        b = x[r:r + step].double().view(-1, x.shape[1] // BLOCK, BLOCK)
        a = b.abs().amax(2, keepdim=True)
        e = torch.floor(torch.log2(a))
        # the logarithm may round across a power of two: compare with the power itself
        e = torch.where(a > 0, e, torch.zeros_like(e))
        e = torch.where(_two_to(e) > a, e - 1, e)
        e = torch.where(_two_to(e + 1) <= a, e + 1, e)
        scale = _two_to(torch.where(a > 0, (e - 2).clamp(-127, 127), torch.full_like(e, -127.0)))
        v = (b.abs() / scale)[..., None]
        d = (v - mags).abs()
        near = d.amin(-1, keepdim=True)
        even = torch.arange(8, device=x.device) % 2
        pick = torch.where(d == near, even, torch.full_like(even, 9).expand(d.shape)).argmin(-1)
        q = torch.copysign(mags[pick] * scale, b)
        out[r:r + step] = q.view(-1, x.shape[1])
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "mx4_quantize":
        return _exact_quant(s["x"])
    if op == "ffn":
        x = s["x"].double()
        gate = torch.einsum("th,ih->ti", x, s["gate_w"].double())
        up = torch.einsum("th,ih->ti", x, s["up_w"].double())
        h = gate * torch.sigmoid(gate) * up
        y = torch.einsum("ti,hi->th", h, s["down_w"].double())
        return {"y": y, "gate": gate, "up": up, "h": h} if case["train"] else {"y": y}
    if op == "ffn_backward":
        dy, gate, up = s["d_y"].double(), s["gate"].double(), s["up"].double()
        sig = torch.sigmoid(gate)
        act, slope = gate * sig, sig + gate * sig * (1 - sig)
        dh = torch.einsum("th,hi->ti", dy, s["down_w"].double())
        dg, du, x = dh * up * slope, dh * act, s["x"].double()
        return (torch.einsum("ti,ih->th", dg, s["gate_w"].double()) + torch.einsum("ti,ih->th", du, s["up_w"].double()),
                torch.einsum("ti,th->ih", dg, x), torch.einsum("ti,th->ih", du, x),
                torch.einsum("th,ti->hi", dy, s["h"].double()))
    if case["form"] == "matmul":
        return torch.einsum("mk,nk->mn", _exact_values(s["a"], s["a_scales"]), _exact_values(s["b"], s["b_scales"]))
    N = case["n"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    a = _exact_values(s["a"], s["a_scales"])
    sizes, starts, offs = s["sizes"].tolist(), s["padded"].tolist(), s["offsets"].tolist()
    for e, n in enumerate(sizes):
        rows = slice(starts[e], starts[e] + n)
        t = slice(e * N // 128, (e + 1) * N // 128)
        c = a[rows] @ _exact_values(s["b"][e], s["b_scales"][t]).t()
        if case["form"] == "gate_up":
            c = c * torch.sigmoid(c) * (a[rows] @ _exact_values(s["b2"][e], s["b2_scales"][t]).t())
        else:
            c = c * s["weights"][offs[e]:offs[e] + n, None].double()
        out[rows] = c
    return out


def work(case):
    op = case["op"]
    if op in ("ffn", "ffn_backward"):
        T, H, I = case["tokens"], case["hidden"], case["inter"]
        if op == "ffn":
            return {"bytes": 2 * (3 * H * I + 2 * T * H + (3 * T * I if case["train"] else 0)), "flops": 6 * T * H * I}
        return {"bytes": 2 * (6 * H * I + 3 * T * H + 3 * T * I), "flops": 12 * T * H * I}
    if op == "mx4_quantize":
        # the values, the codes and scales that stand for them, and the values read back
        n, b = case["rows"] * case["cols"], 4 if case["dtype"] == "fp32" else 2
        return {"bytes": n * (2 * b + 0.5 + 1 / 32), "flops": 2 * n}
    K, N, E = case["k"], case["n"], case["experts"]
    pairs, mats = case["tokens"] * case["top_k"], 2 if case["form"] == "gate_up" else 1
    # experts that some token chose (expected number)
    p = [(e + 1) ** -case["zipf"] for e in range(E)]
    touched = sum(1 - (1 - min(1.0, case["top_k"] * q / sum(p))) ** case["tokens"] for q in p)
    return {"bytes": (pairs * K + mats * touched * N * K) * (0.5 + 1 / 32) + 2 * pairs * N,
            "flops": 2 * mats * pairs * K * N}
