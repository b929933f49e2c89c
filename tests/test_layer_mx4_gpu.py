"""The example layer: a shared expert that learns, and the layer in 4 bits followed
step by step in 64 bits from what the device itself produced."""
import os
import sys

import numpy as np
import pytest
import torch

import mx4_ref
import routed_grouped_gemm_dispatch_gb300 as moe

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer_4bit as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def test_shared_expert_learns():
    """Gradient descent on the squared distance to a teacher goes down every few steps.

    Near the start the loss falls by about lr·|gradient|² per step; over 12 steps the
    last loss has to be below three quarters of the first."""
    torch.manual_seed(0)
    expert = ex.SharedExpert(256, 384, torch.bfloat16, "cuda", seed=1)
    teacher = ex.SharedExpert(256, 384, torch.bfloat16, "cuda", seed=2)
    losses = ex.train_shared_expert(expert, teacher, 256, steps=40, tokens=256)
    assert all(np.isfinite(losses))
    assert np.mean(losses[-5:]) < 0.75 * np.mean(losses[:5]), losses


@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_layer_in_4_bits(tokens, monkeypatch):
    layer = ex.Layer(hidden=256, intermediate=384, experts=8, top_k=2, shared=512, seed=3)
    layer.quantize()
    x = torch.randn((tokens, 256), device="cuda").half()
    seen = []
    for name in ("mx4_quantize", "mx4_gate_up", "mx4_down", "combine_routed"):
        def spy(*a, _f=getattr(moe, name), _n=name, **k):
            r = _f(*a, **k)
            seen.append((_n, a, k, r))
            return r
        monkeypatch.setattr(moe, name, spy)
    y = layer.forward_4bit(x)
    torch.cuda.synchronize()
    assert [s[0] for s in seen] == 2 * ["mx4_quantize", "mx4_gate_up", "mx4_quantize", "mx4_down", "combine_routed"]

    def values(codes, scales, rows):
        c = mx4_ref.unpack(codes.cpu().numpy().reshape(-1, codes.shape[-1]))
        s = mx4_ref.untile(scales.cpu().numpy(), len(c))
        return mx4_ref.values(c, s)[rows]

    def acc(k):
        return (k / 16 + 4) * 2.0 ** -23

    total = np.zeros((tokens, 256))
    for part in (seen[:5], seen[5:]):
        (_, a, k, xq), (_, ga, _, h), (_, ha, hk, hq), (_, da, _, out), (_, ca, _, comb) = part
        rows = k["dest_rows"].cpu().numpy()                       # [T, k]: each token's places
        sizes, padded, gidx = (t.cpu().numpy() for t in ga[6:9])
        valid = np.sort(rows.reshape(-1))
        expert = gidx[valid // 128]
        # every token's codes stand at each of its places
        c, s = mx4_ref.quantize(x.double().cpu().numpy())
        want = mx4_ref.values(c, s)
        for j in range(rows.shape[1]):
            assert np.array_equal(values(xq[0], xq[1], rows[:, j]), want)
        # h from those codes, in 64 bits
        xv = values(xq[0], xq[1], valid)
        E, I = ga[2].shape[:2]
        gw, uw = (values(ga[i], ga[i + 1], slice(None)).reshape(E, I, -1) for i in (2, 4))
        hv = h.double().cpu().numpy()[valid]
        for i, e in enumerate(expert):
            G, U = gw[e] @ xv[i], uw[e] @ xv[i]
            act = G / (1 + np.exp(-G))
            dG, dU = acc(256) * (np.abs(gw[e]) @ np.abs(xv[i])), acc(256) * (np.abs(uw[e]) @ np.abs(xv[i]))
            ref = act * U
            tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2 * (1.1 * np.abs(U) * dG + np.abs(act) * dU + 32 * 2.0 ** -23 * np.abs(ref))
            assert np.all(np.abs(hv[i] - ref) <= tol)
        # the codes of h are those of the device's own h
        c, s = mx4_ref.quantize(hv)
        h4 = mx4_ref.values(c, s)
        assert np.array_equal(values(hq[0], hq[1], valid), h4)
        # down and the routed weights
        dw = values(da[2], da[3], slice(None)).reshape(E, 256, -1)
        w = da[4].double().cpu().numpy()
        offsets = da[6].cpu().numpy()
        ov = out.double().cpu().numpy()[valid]
        for i, e in enumerate(expert):
            rw = w[offsets[e] + valid[i] - padded[e]]
            ref = dw[e] @ h4[i] * rw
            tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2 * acc(I) * (np.abs(dw[e]) @ np.abs(h4[i])) * rw + 2.0 ** -23 * np.abs(ref)
            assert np.all(np.abs(ov[i] - ref) <= tol)
        total += comb.double().cpu().numpy()
    # the sum of the two parts, in fp16
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got - total) <= 2.0 ** -11 * np.abs(total) + 2.0 ** -25)
