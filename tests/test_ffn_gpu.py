"""The dense gated feed-forward block and its gradients against the formulas in 64 bits.

Every stage is compared with the formula applied to what the device itself fed
into it, so that each tolerance is one rounding to the output type (half a step,
eps/2 relative, plus half of fp16's smallest subnormal) and the error of an fp32
sum: the tensor cores add 16 products at a time, so a sum over K has K/16 + a few
additions, each off by at most 2^-23 of the sum of the absolute products.
"""
import numpy as np
import pytest
import torch

import routed_grouped_gemm_dispatch_gb300 as moe

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16]
# tokens, hidden, intermediate: one row and tile edges in every direction, smallest widths
SHAPES = [(1, 8, 8), (3, 16, 24), (1, 256, 384), (2, 136, 264), (7, 512, 136), (31, 264, 520), (32, 128, 128),
          (33, 1024, 256), (63, 264, 392), (64, 256, 1032), (65, 520, 136), (127, 256, 128), (128, 128, 256),
          (129, 384, 640), (255, 520, 264), (257, 128, 1288), (300, 2048, 408), (513, 776, 512), (1025, 256, 264),
          # few tiles and a long K axis: tiles shared by two and four pairs
          (260, 520, 2056), (520, 1544, 1288), (200, 4104, 136)]


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    return 2.0 ** -25 if dt == torch.float16 else 0.0


def acc(k):
    return (k / 16 + 4) * 2.0 ** -23


def rounding(ref, dt):
    return half_step(dt) * ref.abs() + tiny(dt)


def check(got, ref, tol, what):
    assert got.shape == ref.shape
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - tol).max()):.3e}"


def make(T, H, I, dt, seed=0):
    """Inputs as leading rows of larger buffers whose other rows are NaN: a read past T would show."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rows(n, cols, std=1.0):
        buf = torch.full((n + 130, cols), float("nan"), dtype=dt, device="cuda")
        buf[:n] = torch.randn((n, cols), generator=g, device="cuda").mul_(std).to(dt)
        return buf[:n]

    return {"x": rows(T, H), "gate_w": rows(I, H, H ** -0.5), "up_w": rows(I, H, H ** -0.5),
            "down_w": rows(H, I, I ** -0.5), "d_out": rows(T, H)}


def guarded(T, cols, dt):
    """A buffer of T rows inside a larger one filled with a pattern that must survive."""
    buf = torch.full((T + 129, cols), 0x7D5A, dtype=torch.int16, device="cuda").view(dt)
    return buf, buf[:T]


def untouched(buf, T):
    return bool((buf[T:].view(torch.int16) == 0x7D5A).all())


def silu64(g):
    return g * torch.sigmoid(g)


def check_forward(m, h, gate, up, out, dt):
    x, wg, wu, wd = (m[k].double() for k in ("x", "gate_w", "up_w", "down_w"))
    H, I = wd.shape
    G, U = x @ wg.t(), x @ wu.t()
    dG, dU = acc(H) * (x.abs() @ wg.abs().t()), acc(H) * (x.abs() @ wu.abs().t())
    if gate is not None:
        check(gate, G, rounding(G, dt) + 2 * dG, "gate")
        check(up, U, rounding(U, dt) + 2 * dU, "up")
    ref = silu64(G) * U
    # |silu'| <= 1.1; the exponential and the quotient: 32 steps of fp32
    off = 1.1 * U.abs() * dG + silu64(G).abs() * dU + 1.1 * dG * dU + 32 * 2.0 ** -23 * ref.abs()
    check(h, ref, rounding(ref, dt) + 2 * off, "up_logits")
    hd = h.double()
    y = hd @ wd.t()
    check(out, y, rounding(y, dt) + 2 * acc(I) * (hd.abs() @ wd.abs().t()), "out")


@pytest.mark.parametrize("dt", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("T,H,I", SHAPES)
def test_forward(T, H, I, dt):
    m = make(T, H, I, dt, seed=T)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bufs = {k: guarded(T, c, dt) for k, c in (("out", H), ("up_logits", I), ("gate", I), ("up", I))}
    got = moe.gated_ffn(m["x"], m["gate_w"], m["up_w"], m["down_w"], status=status,
                        **{k: v[1] for k, v in bufs.items()})
    plain = moe.gated_ffn(m["x"], m["gate_w"], m["up_w"], m["down_w"], status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert got.data_ptr() == bufs["out"][1].data_ptr()
    for k, (buf, _) in bufs.items():
        assert untouched(buf, T), k
    check_forward(m, bufs["up_logits"][1], bufs["gate"][1], bufs["up"][1], got, dt)
    assert torch.equal(plain.view(torch.int16), got.view(torch.int16))      # storing gate and up changes nothing


def stored(m, dt):
    T, I = m["x"].shape[0], m["gate_w"].shape[0]
    s = {k: torch.empty((T, I), dtype=dt, device="cuda") for k in ("gate", "up", "up_logits")}
    moe.gated_ffn(m["x"], m["gate_w"], m["up_w"], m["down_w"], **s)
    return s


@pytest.mark.parametrize("dt", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("T,H,I", SHAPES)
def test_backward(T, H, I, dt):
    m = make(T, H, I, dt, seed=1000 + T)
    s = stored(m, dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.ffn_backward_workspace_bytes(T, I), dtype=torch.uint8, device="cuda")
    bufs = {"d_x": guarded(T, H, dt), "d_gate_w": guarded(I, H, dt), "d_up_w": guarded(I, H, dt),
            "d_down_w": guarded(H, I, dt)}
    args = (m["d_out"], m["x"], m["gate_w"], m["up_w"], m["down_w"], s["gate"], s["up"], s["up_logits"])
    got = moe.gated_ffn_backward(*args, workspace=ws, status=status, **{k: v[1] for k, v in bufs.items()})
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for (k, (buf, part)), t in zip(bufs.items(), got):
        assert t.data_ptr() == part.data_ptr() and untouched(buf, part.shape[0]), k

    half = ws.numel() // 2
    dG = ws[:T * I * 2].view(dt).view(T, I)
    dU = ws[half:half + T * I * 2].view(dt).view(T, I)
    dy, x, wg, wu, wd = (m[k].double() for k in ("d_out", "x", "gate_w", "up_w", "down_w"))
    g, u, h = s["gate"].double(), s["up"].double(), s["up_logits"].double()
    dh, ddh = dy @ wd, 2 * acc(H) * (dy.abs() @ wd.abs())
    sg = torch.sigmoid(g)
    slope = sg * (1 + g * (1 - sg))
    # 1 + g(1 - s) may cancel: its error goes by the terms' sizes; 16 steps of fp32
    size = sg * (1 + 2 * g.abs())
    ref = dh * u * slope
    check(dG, ref, rounding(ref, dt) + 1.1 * u.abs() * ddh + 2.0 ** -19 * (dh * u).abs() * size, "d_G")
    ref = dh * g * sg
    check(dU, ref, rounding(ref, dt) + (g * sg).abs() * ddh + 2.0 ** -19 * ref.abs(), "d_U")
    dGd, dUd = dG.double(), dU.double()

    def product(got, parts, k, what):
        ref = sum(a @ b for a, b in parts)
        tol = rounding(ref, dt) + 2 * acc(k) * sum(a.abs() @ b.abs() for a, b in parts)
        check(got, ref, tol, what)

    product(got[0], [(dGd, wg), (dUd, wu)], 2 * I + 128, "d_x")
    product(got[1], [(dGd.t(), x)], T, "d_gate_w")
    product(got[2], [(dUd.t(), x)], T, "d_up_w")
    product(got[3], [(dy.t(), h)], T, "d_down_w")

    fresh = moe.gated_ffn_backward(*args)
    torch.cuda.synchronize()
    for a, b in zip(fresh, got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("dt", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("T,H,I", [(520, 512, 3336), (1025, 904, 2056), (900, 640, 2560), (448, 384, 7176),
                                   (33, 512, 1024), (32, 1032, 776), (24, 2048, 520), (400, 768, 2048),
                                   (257, 4096, 520)])
def test_backward_where_the_launches_differ(T, H, I, dt):
    """More tiles of d_h than one shared round (d_down joins the first launch) or fewer; boxes of
    few rows; pairs without a shared tile ahead of the others."""
    test_backward(T, H, I, dt)


@pytest.mark.parametrize("dt", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("T,H,I", [(5, 64, 72), (130, 72, 136)])
def test_gradients_against_differences(T, H, I, dt):
    """Σ d_out ⊙ out in 64 bits, differenced along each gradient's own direction.

    Along its own unit direction a gradient g has the slope |g|.  The device's
    is off by a few roundings (stored gate and up, h, d_G or d_U, the result),
    each at most a half step of |g| in the 2-norm: eight half steps are allowed,
    and 1e-6 for the difference quotient (third derivatives, step 1e-4)."""
    m = make(T, H, I, dt, seed=7)
    s = stored(m, dt)
    got = moe.gated_ffn_backward(m["d_out"], m["x"], m["gate_w"], m["up_w"], m["down_w"], s["gate"], s["up"],
                                 s["up_logits"])
    names = ("x", "gate_w", "up_w", "down_w")
    p = {k: m[k].double() for k in names}
    dy = m["d_out"].double()

    def loss(q):
        return float(((silu64(q["x"] @ q["gate_w"].t()) * (q["x"] @ q["up_w"].t())) @ q["down_w"].t() * dy).sum())

    for name, g in zip(names, got):
        g = g.double()
        n = float(g.norm())
        v = g / n
        eps = 1e-4
        slope = (loss({**p, name: p[name] + eps * v}) - loss({**p, name: p[name] - eps * v})) / (2 * eps)
        assert abs(slope - n) <= (8 * half_step(dt) + 1e-6) * n, (name, slope, n)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_a_bad_row_stays_in_its_row(T):
    """NaN and infinity in one token's input do not reach another token's output."""
    m = make(T + 2, 256, 264, torch.bfloat16, seed=5)
    want = moe.gated_ffn(m["x"], m["gate_w"], m["up_w"], m["down_w"])
    x = m["x"].clone()
    x[T // 2, 3] = float("nan")
    x[T + 1, 250] = float("inf")
    got = moe.gated_ffn(x, m["gate_w"], m["up_w"], m["down_w"])
    torch.cuda.synchronize()
    keep = [t for t in range(T + 2) if t not in (T // 2, T + 1)]
    assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16))
    assert bool(got[T // 2].isnan().all()) and not bool(got[T + 1].isfinite().any())


def test_saturated_gates():
    """Gates far out on both sides: silu is the identity or zero, its slope one or zero."""
    dt, T, H, I = torch.bfloat16, 4, 8, 16
    x = torch.zeros((T, H), dtype=dt, device="cuda")
    x[:, 0] = torch.tensor([200.0, -200.0, 95.0, -95.0], dtype=dt)
    x[:, 1] = 1.0
    gate_w = torch.zeros((I, H), dtype=dt, device="cuda")
    up_w = torch.zeros((I, H), dtype=dt, device="cuda")
    gate_w[:, 0] = 1.0
    up_w[:, 1] = 2.0
    down_w = torch.eye(H, I, dtype=dt, device="cuda")
    s = {k: torch.empty((T, I), dtype=dt, device="cuda") for k in ("gate", "up", "up_logits")}
    out = moe.gated_ffn(x, gate_w, up_w, down_w, **s)
    dy = torch.ones((T, H), dtype=dt, device="cuda")
    d_x, d_g, d_u, d_d = moe.gated_ffn_backward(dy, x, gate_w, up_w, down_w, s["gate"], s["up"], s["up_logits"])
    torch.cuda.synchronize()
    gate = x[:, :1].float()
    want = torch.where(gate > 0, 2 * gate, torch.zeros_like(gate)).expand(T, H)
    assert torch.equal(out.float(), want)
    for t in (d_x, d_g, d_u, d_d):
        assert bool(t.isfinite().all())
    # d_x: the gate's slope times up (2), and 2 silu(gate) for the up input, over H outputs
    assert torch.equal(d_x[:, 0].float(), torch.where(gate[:, 0] > 0, 2.0 * H, 0.0))


def test_no_tokens():
    dt = torch.float16
    m = make(1, 128, 136, dt)
    x = m["x"][:0]
    out = moe.gated_ffn(x, m["gate_w"], m["up_w"], m["down_w"])
    assert out.shape == (0, 128)
    e = torch.empty((0, 136), dtype=dt, device="cuda")
    d_x, *dw = moe.gated_ffn_backward(x, x, m["gate_w"], m["up_w"], m["down_w"], e, e, e)
    torch.cuda.synchronize()
    assert d_x.shape == (0, 128)
    for t in dw:
        assert bool((t == 0).all())


@pytest.mark.parametrize("T", [3, 200])
def test_streams_and_graph_capture(T):
    """The same bits on another stream and from a captured graph, forward and backward in one."""
    dt = torch.bfloat16
    m = make(T, 264, 392, dt, seed=11)
    s = stored(m, dt)
    ws = torch.empty(moe.ffn_backward_workspace_bytes(T, 392), dtype=torch.uint8, device="cuda")
    bufs = {k: torch.empty_like(v) for k, v in (("out", m["x"]), ("d_x", m["x"]), ("d_gate_w", m["gate_w"]),
                                                 ("d_up_w", m["up_w"]), ("d_down_w", m["down_w"]))}

    def step():
        moe.gated_ffn(m["x"], m["gate_w"], m["up_w"], m["down_w"], out=bufs["out"], **s)
        moe.gated_ffn_backward(m["d_out"], m["x"], m["gate_w"], m["up_w"], m["down_w"], s["gate"], s["up"],
                               s["up_logits"], workspace=ws, **{k: bufs[k] for k in bufs if k != "out"})

    step()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in bufs.items()}
    side = torch.cuda.Stream()
    for v in bufs.values():
        v.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    for k in bufs:
        assert torch.equal(bufs[k].view(torch.int16), want[k].view(torch.int16)), k
        bufs[k].zero_()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for k in bufs:
        assert torch.equal(bufs[k].view(torch.int16), want[k].view(torch.int16)), k


def test_refusals():
    """What the checks name: types, shapes, strides, half of what is stored, a short workspace."""
    dt = torch.float16
    m = make(3, 16, 24, dt)
    w = (m["gate_w"], m["up_w"], m["down_w"])
    e = torch.empty((3, 24), dtype=dt, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        moe.gated_ffn(torch.empty((16, 3), dtype=dt, device="cuda").t(), *w)
    with pytest.raises(TypeError, match="gate_w"):
        moe.gated_ffn(m["x"], w[0].bfloat16(), *w[1:])
    with pytest.raises(ValueError, match="up_w"):
        moe.gated_ffn(m["x"], w[0], w[1][:8], w[2])
    with pytest.raises(ValueError, match="down_w"):
        moe.gated_ffn(m["x"], w[0], w[1], w[1])
    with pytest.raises(ValueError, match="both or neither"):
        moe.gated_ffn(m["x"], *w, gate=e)
    with pytest.raises(ValueError, match="out"):
        moe.gated_ffn(m["x"], *w, out=e)
    with pytest.raises(ValueError, match="2 dims"):
        moe.gated_ffn(m["x"][0], *w)
    with pytest.raises(moe.MoeError, match="MOE_ERR_SHAPE"):
        odd = torch.zeros((3, 12), dtype=dt, device="cuda")
        moe.gated_ffn(odd, odd, odd, torch.zeros((12, 3), dtype=dt, device="cuda"))
    with pytest.raises(ValueError, match="d_out"):
        moe.gated_ffn_backward(e, m["x"], *w, e, e, e)
    with pytest.raises(moe.MoeError, match="MOE_ERR_WORKSPACE"):
        moe.gated_ffn_backward(m["x"], m["x"], *w, e, e, e, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(moe.MoeError, match="MOE_ERR_ALIGN"):
        moe.gated_ffn(m["x"], *w, up_logits=torch.empty(3 * 24 + 1, dtype=dt, device="cuda")[1:].view(3, 24))


@pytest.mark.parametrize("T", [2, 200])
def test_own_buffers_on_a_given_stream(T):
    """Buffers that the calls allocate themselves hold until the given stream is done with them."""
    dt = torch.bfloat16
    m = make(T, 264, 392, dt, seed=21)
    s = stored(m, dt)
    args = (m["d_out"], m["x"], m["gate_w"], m["up_w"], m["down_w"], s["gate"], s["up"], s["up_logits"])
    want = (moe.gated_ffn(*args[1:5]), *moe.gated_ffn_backward(*args))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = []
        for _ in range(8):
            got.append((moe.gated_ffn(*args[1:5], stream=stream), *moe.gated_ffn_backward(*args, stream=stream)))
            # other work on the current stream that would take a freed buffer
            torch.full((T, 392), float("nan"), dtype=dt, device="cuda")
            torch.full((moe.ffn_backward_workspace_bytes(T, 392),), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for g in got:
            for a, b in zip(g, want):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31: the last rows' results are those of a call on them alone,
    and the weights' gradients are the sum of those of two halves."""
    dt, T, H, I = torch.bfloat16, 280_001, 8, 8192
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn((T, H), generator=g, device="cuda").to(dt)
    d_out = torch.randn((T, H), generator=g, device="cuda").to(dt)
    w = [torch.randn((I, H), generator=g, device="cuda").to(dt) for _ in range(2)]
    w.append((torch.randn((H, I), generator=g, device="cuda") * I ** -0.5).to(dt))
    s = {k: torch.empty((T, I), dtype=dt, device="cuda") for k in ("gate", "up", "up_logits")}
    out = moe.gated_ffn(x, *w, **s)
    d_x, *dw = moe.gated_ffn_backward(d_out, x, *w, s["gate"], s["up"], s["up_logits"])
    # from the last full tile of 256 rows on, so that the rows sit alike in their tiles
    at = T // 256 * 256 - 256
    assert at * I > 2 ** 31
    t = {k: torch.empty((T - at, I), dtype=dt, device="cuda") for k in s}
    want = moe.gated_ffn(x[at:], *w, **t)
    want_x = moe.gated_ffn_backward(d_out[at:], x[at:], *w, t["gate"], t["up"], t["up_logits"])[0]
    tail = (x[at:].double() @ w[0].double().t(), x[at:].double() @ w[1].double().t())
    check(s["gate"][at:], tail[0], rounding(tail[0], dt) + 2 * acc(H) * (x[at:].double().abs() @ w[0].double().abs().t()), "gate")
    check(s["up"][at:], tail[1], rounding(tail[1], dt) + 2 * acc(H) * (x[at:].double().abs() @ w[1].double().abs().t()), "up")
    # the two calls may split their sums differently: an fp32 sum and one rounding apart
    y = t["up_logits"].double() @ w[2].double().t()
    tol = 2 * rounding(y, dt) + 4 * acc(I) * (t["up_logits"].double().abs() @ w[2].double().abs().t())
    # up_logits of the two calls differ by a rounding where an fp32 sum fell on either side of it
    tol = tol + 2 * half_step(dt) * (t["up_logits"].double().abs() @ w[2].double().abs().t())
    check(out[at:], want.double(), tol, "out")
    assert float((d_x[at:].double() - want_x.double()).norm()) <= 8 * half_step(dt) * float(want_x.double().norm())
    # gradients of the weights: two halves added in fp32, each rounded once
    half = T // 2
    parts = [moe.gated_ffn_backward(d_out[a:b], x[a:b], *w, s["gate"][a:b], s["up"][a:b], s["up_logits"][a:b])[1:]
             for a, b in ((0, half), (half, T))]
    for got, p, q in zip(dw, *parts):
        ref = p.double() + q.double()
        tol = half_step(dt) * (p.double().abs() + q.double().abs() + 2 * ref.abs())
        err = (got.double() - ref).norm()
        # (a random walk's partial sums are about as large as its end: acc(T) of it for the fp32 sum)
        assert float(err) <= float(tol.norm()) + acc(T) * float(got.double().norm())
