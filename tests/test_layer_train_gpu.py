"""The training operators together, as a step of a routed layer uses them: routing with its logits, experts and shared
expert forward, gradients of the router from the layer's own output and from the losses, gradients of
the shared expert, and orthogonalised updates; each followed in 64 bits from what the device itself produced."""
import os
import sys

import numpy as np
import pytest
import torch

import routed_grouped_gemm_dispatch_gb300 as moe
import test_ortho_gpu as ortho
import test_router_train_gpu as router

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer_4bit as ex  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,seqs,masked", [(64, 1, False), (300, 3, True)])
def test_a_training_step(tokens, seqs, masked):
    T, H, I, E, k = tokens, 256, 384, 12, 3
    layer = ex.Layer(hidden=H, intermediate=I, experts=E, top_k=k, shared=512, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn((T, H), generator=g, device="cuda").half()
    target = torch.randn((T, H), generator=g, device="cuda").half()
    s = {"mask": None, "offs": None}
    if seqs > 1:
        s["offs"] = torch.tensor([0, T // 4, T // 2, T], dtype=torch.int32, device="cuda")
    if masked:
        s["mask"] = torch.rand((T,), generator=g, device="cuda") >= 0.1
    kw = dict(token_mask=s["mask"], seq_offsets=s["offs"])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    # forward
    s["z"] = torch.empty((T, E), device="cuda")
    s["ids"], weights = moe.router_topk(x, layer.router_w, k, logits=s["z"], status=status)
    tables = moe.build_dispatch(s["ids"], E, status=status)
    rows = tables["group_idx_for_bx"].numel() * moe.BLOCK_TOKEN
    packed = moe.pack_routed(s["ids"], weights, x, tables, rows, status=status)
    h, out = torch.empty((rows, I), dtype=x.dtype, device="cuda"), torch.empty((rows, H), dtype=x.dtype, device="cuda")
    moe.fused_forward(packed["stacked_expert_tokens"], layer.gate_w, layer.up_w, layer.down_w, packed["routed_expert_weights"],
                      tables["group_sizes"], tables["group_offsets"], tables["group_padded_offsets"],
                      tables["group_idx_for_bx"], h, out, status=status)
    y = moe.combine_routed(out, packed["pair_padded_rows"]) + layer.shared.forward(x, train=True)
    losses, counts, seq_tokens = moe.router_balance(s["z"], s["ids"], status=status, **kw)
    # the counts are the dispatch table's, where every token counts
    if not masked:
        assert torch.equal(counts.sum(0).to(torch.int32), tables["group_sizes"])
    want, c, n, tol = router.reference(s)
    assert np.array_equal(counts.cpu().numpy(), c) and np.all(np.abs(losses.double().cpu().numpy() - want) <= tol)

    # backward: of a squared distance, times a loss scale; masked tokens have none
    d_y = ((y.float() - target.float()) * (64.0 / T)).half()
    if masked:
        d_y[~s["mask"]] = 0
    # a routed weight multiplies its expert's row: its gradient is the row without it, by the output's gradient
    pairs = out[packed["pair_padded_rows"].long()].float() / weights[..., None]
    d_w = torch.einsum("tkh,th->tk", pairs, d_y.float()).contiguous()
    d_losses = torch.tensor([0.64, 0.064], device="cuda")
    d_z = torch.empty_like(s["z"])
    d_x, d_router = moe.router_backward(x, layer.router_w, s["z"], s["ids"], d_w, d_losses, counts, seq_tokens, d_logits=d_z,
                                        status=status, **kw)
    router.check_grads(s, x, layer.router_w, d_w, d_losses, (d_x, d_router), d_z, c, n)
    d_x2, *shared = layer.shared.backward(d_y)
    assert torch.isfinite(d_x.float() + d_x2.float()).all()
    torch.cuda.synchronize()
    assert int(status) == 0

    # updates, singly and as a stack: gate and up have one shape
    stack = torch.stack(shared[:2])
    updates = moe.orthogonalize(stack, status=status)
    for i in range(2):
        assert torch.equal(updates[i], moe.orthogonalize(shared[i]))
    ortho.check(stack, updates)
    ortho.check(d_router, moe.orthogonalize(d_router, status=status))
    ortho.check(shared[2], moe.orthogonalize(shared[2], status=status))
    assert int(status) == 0


def test_gradients_of_the_losses_against_differences():
    """The example's balance step: its gradient against differences of the loss that the library itself reports, with the
    ids held (the counts are constants in the gradient)."""
    T, H, E, k = 256, 256, 16, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn((T, H), generator=g, device="cuda").half()
    w = torch.randn((E, H), generator=g, device="cuda").mul_(H ** -0.5).half()
    _, counts, d_w = ex.balance_step(x, w, k, balance_weight=1.0, z_weight=0.5)
    ids, _ = moe.router_topk(x, w, k)
    xd = x.double()

    def loss(weights):
        z = (xd @ weights.t()).float().contiguous()
        bal, _, _ = moe.router_balance(z, ids)
        return float(bal[0].double() + 0.5 * bal[1].double())

    direction = torch.randn((E, H), generator=g, device="cuda").double() * H ** -0.5
    eps = 2.0 ** -6
    diff = (loss(w.double() + eps * direction) - loss(w.double() - eps * direction)) / (2 * eps)
    got = float((d_w.double() * direction).sum())
    # differences: eps² / 6 of a third derivative (below 4 times the loss's size here), the losses' rounding
    # 2^-22 of them over eps; the gradient: two roundings of 2^-11 of the terms' sizes
    size = loss(w.double())
    terms = float((d_w.double().abs() * direction.abs()).sum())
    assert abs(got - diff) <= eps ** 2 / 6 * 4 * size + 2.0 ** -22 * size / eps + 2.0 ** -10 * terms


def test_router_training_runs():
    layer = ex.Layer(hidden=256, intermediate=384, experts=8, top_k=2, shared=512, seed=3)
    x = torch.randn((500, 256), device="cuda").half()
    losses = ex.train_router(layer, x, steps=5)
    assert len(losses) == 5 and np.isfinite(losses).all() and torch.isfinite(layer.router_w).all()
    expert = ex.SharedExpert(256, 384, torch.bfloat16, "cuda", seed=1)
    teacher = ex.SharedExpert(256, 384, torch.bfloat16, "cuda", seed=2)
    losses = ex.train_shared_expert(expert, teacher, 256, steps=3, tokens=256, lr=0.02, orthogonal=True)
    assert np.isfinite(losses).all()
