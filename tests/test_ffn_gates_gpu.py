"""The activation and its slope over gates from far below to far above zero, on the kernel of few
tokens and on the tiles, against the formulas in 64 bits.

Gates, up values and incoming gradients are exact in every type and reach the epilogue through
products with a single term, so only the epilogue is compared.  The sigmoid is off by the rounding
of x·log2 e before the power (2^-24 of it and of the constant, at most 2^-23.7 |x| of the result
together), the power (2^-22), the sum (2^-24) and the reciprocal (2^-23), less than 2^-23.7 |x| +
2^-21 in all, and is 0 where it would be below 2^-126.
"""
import pytest
import torch

import routed_grouped_gemm_dispatch_gb300 as moe

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16]
UP, DY = 1.25, 0.75


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    return 2.0 ** -25 if dt == torch.float16 else 2.0 ** -134


def sigmoid_error(g):
    return 2.0 ** -23.7 * g.abs() + 2.0 ** -21


def inputs(gates, dt):
    T, H, I = gates.numel(), 8, 16
    x = torch.zeros((T, H), dtype=dt, device="cuda")
    x[:, 0], x[:, 1] = gates, 1.0
    gate_w, up_w = torch.zeros((I, H), dtype=dt, device="cuda"), torch.zeros((I, H), dtype=dt, device="cuda")
    gate_w[:, 0], up_w[:, 1] = 1.0, UP
    return x, gate_w, up_w, torch.eye(H, I, dtype=dt, device="cuda")


def check(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} off, worst at gate {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("dt", DTYPES, ids=["fp16", "bf16"])
@pytest.mark.parametrize("T", [128, 129, 1000])
def test_gates_far_out(T, dt):
    lo, hi = (-110.0, 110.0) if dt == torch.bfloat16 else (-20.0, 20.0)     # (fp16 holds nothing of silu below -20)
    near = torch.linspace(-4.0, 4.0, T // 4, dtype=torch.float64)
    gates = torch.cat([near, torch.linspace(lo, hi, T - T // 4, dtype=torch.float64)]).to(dt).cuda()
    x, gate_w, up_w, down_w = inputs(gates, dt)
    s = {k: torch.empty((T, 16), dtype=dt, device="cuda") for k in ("gate", "up", "up_logits")}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = moe.gated_ffn(x, gate_w, up_w, down_w, status=status, **s)
    d_y = torch.full((T, 8), DY, dtype=dt, device="cuda")
    ws = torch.empty(moe.ffn_backward_workspace_bytes(T, 16), dtype=torch.uint8, device="cuda")
    moe.gated_ffn_backward(d_y, x, gate_w, up_w, down_w, s["gate"], s["up"], s["up_logits"], workspace=ws, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert bool((s["gate"] == gates[:, None]).all()) and bool((s["up"] == UP).all())
    assert torch.equal(out, s["up_logits"][:, :8])

    g = gates.double()[:, None].expand(T, 16)
    sg, rel, flush = torch.sigmoid(g), sigmoid_error(g), 2.0 ** -126
    ref = g * sg * UP
    tol = (half_step(dt) + rel + 4 * 2.0 ** -24) * ref.abs() + flush * (g * UP).abs() + tiny(dt)
    check(s["up_logits"], ref, tol, "up_logits")

    half = ws.numel() // 2
    dG, dU = (ws[at:at + T * 32].view(dt).view(T, 16)[:, :8] for at in (0, half))
    g, sg, rel = g[:, :8], sg[:, :8], rel[:, :8]
    ref = DY * g * sg
    check(dU, ref, (half_step(dt) + rel + 4 * 2.0 ** -24) * ref.abs() + flush * (DY * g).abs() + tiny(dt), "d_U")
    slope = 1 + g * (1 - sg)
    ref = DY * UP * sg * slope
    # the slope's own terms: 1 - s (an error of s, and a rounding), its product and the sum
    own = g.abs() * (sg * rel + 3 * 2.0 ** -24 * (1 - sg)) + 2.0 ** -24 * slope.abs()
    tol = ((half_step(dt) + rel + 4 * 2.0 ** -24) * ref.abs() + DY * UP * sg * own * (1 + rel)
           + flush * DY * UP * (1 + g.abs()) + tiny(dt))
    check(dG, ref, tol, "d_G")


@pytest.mark.parametrize("T", [8, 130, 400])
def test_saturated_gates(T):
    """Far out on both sides silu is the identity or zero and its slope one or zero, to the bit."""
    dt = torch.bfloat16
    far = torch.tensor([200.0, -200.0, 112.0, -112.0, 3e4, -3e4, 1e30, -1e30], dtype=torch.float64)
    gates = far.repeat(-(-T // 8))[:T].to(dt).cuda()
    x, gate_w, up_w, down_w = inputs(gates, dt)
    s = {k: torch.empty((T, 16), dtype=dt, device="cuda") for k in ("gate", "up", "up_logits")}
    moe.gated_ffn(x, gate_w, up_w, down_w, **s)
    d_y = torch.full((T, 8), DY, dtype=dt, device="cuda")
    ws = torch.empty(moe.ffn_backward_workspace_bytes(T, 16), dtype=torch.uint8, device="cuda")
    moe.gated_ffn_backward(d_y, x, gate_w, up_w, down_w, s["gate"], s["up"], s["up_logits"], workspace=ws)
    torch.cuda.synchronize()
    on = gates[:, None] > 0
    zero = torch.zeros((), device="cuda")
    assert torch.equal(s["up_logits"].float(), torch.where(on, (gates.float() * UP).to(dt).float()[:, None], zero).expand(T, 16))
    half = ws.numel() // 2
    dG, dU = (ws[at:at + T * 32].view(dt).view(T, 16)[:, :8].float() for at in (0, half))
    assert torch.equal(dU, torch.where(on, (gates.float() * DY).to(dt).float()[:, None], zero).expand(T, 8))
    assert torch.equal(dG, torch.where(on, torch.tensor(DY * UP, device="cuda").to(dt).float(), zero).expand(T, 8))
