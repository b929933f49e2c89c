"""The router's losses and gradients where neighbouring tokens share experts, with peaked logits, and at sizes and tables
that the other tests leave out; against the formulas in 64 bits, with the tolerances of test_router_train_gpu unless
a test derives its own."""
import pytest
import torch

import routed_grouped_gemm_dispatch_gb300 as moe
import test_router_train_gpu as router

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,seqs", [(3000, 64, 4, 1), (3000, 128, 8, 900), (1300, 256, 16, 1), (1300, 130, 3, 400),
                                        (700, 700, 8, 200), (2100, 9, 9, 700)])
def test_neighbouring_tokens_share_experts(T, E, k, seqs, dtype):
    """One token's routed gradients are gone from its experts before the next token's are there: every token names
    the same experts, in another order, and sequences of two or three tokens change the counts under them."""
    s = router.make(T, E, k, seqs, seed=T + E)
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    order = torch.rand((T, k), generator=g, device="cuda").argsort(dim=1)
    s["ids"] = order.mul(max(1, E // k)).to(torch.int32).contiguous()
    x = torch.randn((T, 64), generator=g, device="cuda").to(dtype)
    w = torch.randn((E, 64), generator=g, device="cuda").to(dtype)
    dw = torch.randn((T, k), generator=g, device="cuda") * 4
    dl = torch.tensor([8.0, 0.5], device="cuda")
    kw = dict(seq_offsets=s["offs"])
    _, counts, tokens = moe.router_balance(s["z"], s["ids"], **kw)
    c, n = counts.cpu().numpy(), tokens.cpu().numpy()
    for a, b in ((dw, None), (dw, dl)):
        d_logits = torch.empty((T, E), device="cuda")
        got = moe.router_backward(x, w, s["z"], s["ids"], a, b, counts if b is not None else None,
                                  tokens if b is not None else None, d_logits=d_logits, **kw)
        router.check_grads(s, x, w, a, b, got, d_logits, c, n)
        for _ in range(5):
            again = torch.empty_like(d_logits)
            moe.router_backward(x, w, s["z"], s["ids"], a, b, counts if b is not None else None,
                                tokens if b is not None else None, d_logits=again, **kw)
            assert torch.equal(again, d_logits)


@pytest.mark.parametrize("T,E,seqs", [(5, 12, 1), (700, 64, 3), (40000, 64, 2), (2000, 1000, 40)])
def test_a_row_of_lowest_values(T, E, seqs):
    """Its logsumexp squared is beyond fp32: the z loss is infinite, as the formula's is once rounded, and nothing else is."""
    s = router.make(T, E, 2, seqs, seed=T)
    s["z"][T // 2] = torch.finfo(torch.float32).min
    losses, counts, tokens = moe.router_balance(s["z"], s["ids"], seq_offsets=s["offs"])
    want, c, n, tol = router.reference(s)
    assert want[1] > 1e70 and float(losses[1]) == float("inf")
    assert abs(float(losses[0]) - want[0]) <= tol[0]
    assert (counts.cpu().numpy() == c).all() and (tokens.cpu().numpy() == n).all()


BAD_OFFSETS = [[0, 60, 30, 100], [0, 101], [-1, 100], [0, 2 ** 31 - 1], [-2 ** 31, 50, 100]]


@pytest.mark.parametrize("offs", BAD_OFFSETS + [list(range(0, 90, 2)) + [80, 100]])
def test_bad_offsets_are_reported_by_both(offs):
    """By the losses in one launch (few sequences) and in two, and by the gradients."""
    T, E, k = 100, 32, 4
    for extra in (0, 20000):
        s = router.make(T + extra, E, k, seed=2)
        o = torch.tensor([v + extra if v >= 0 and v < 2 ** 31 - 1 and i == len(offs) - 1 else v for i, v in enumerate(offs)],
                         dtype=torch.int32, device="cuda")
        x, w = torch.zeros((T + extra, 8), device="cuda").half(), torch.zeros((E, 8), device="cuda").half()
        dw = torch.zeros((T + extra, k), device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        _, counts, tokens = moe.router_balance(s["z"], s["ids"], seq_offsets=o, status=status)
        assert int(status) == moe.MOE_DEV_BAD_TABLE
        status.zero_()
        moe.router_backward(x, w, s["z"], s["ids"], dw, seq_offsets=o, status=status)
        assert int(status) == moe.MOE_DEV_BAD_TABLE


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), 3.4e38])
@pytest.mark.parametrize("T", [200, 5000])
def test_one_gradient_that_is_not_finite(T, bad):
    """The other tokens' gradients are as exact beside it as they are without, in fp16 too."""
    E, k, H = 64, 6, 256
    s = router.make(T, E, k, seed=4)
    x, w = torch.randn((T, H), device="cuda").half(), (torch.randn((E, H), device="cuda") * 1e3).half()
    dw = torch.randn((T, k), device="cuda") * 1e-7
    hit = T // 2
    dw[hit, 1] = bad
    d_x, _ = moe.router_backward(x, w, s["z"], s["ids"], dw)
    assert not torch.isfinite(d_x[hit].float()).any()
    others = torch.arange(T, device="cuda") != hit
    part = {"z": s["z"][others], "ids": s["ids"][others], "mask": None, "offs": None}
    dz, tol = router.grads_reference(part, dw[others].double().cpu().numpy(), None, None, [T - 1, T - 1])
    largest = abs(dz).max()
    if bad == 3.4e38:                   # finite, and so one of those that the common power of two is for
        largest = abs(router.grads_reference(s, dw.double().cpu().numpy(), None, None, [T, T])[0]).max()
    # d_z as an operand: in two terms up to 2048 tokens, one rounding beyond, and half of fp16's least step, 2^-25, where the
    # largest is at 2^13 at least, 2^-38 of it; then 64 products, d_x's own rounding and its least step
    r, wv = 2.0 ** -11, w.double().cpu().numpy()
    want = dz @ wv
    dz_tol = tol + ((r if T > 2048 else r * r) + 2.0 ** -23) * (abs(dz) + tol) + largest * 2.0 ** -38
    bound = dz_tol @ abs(wv) + (2 * E / 16 + 8) * 2.0 ** -23 * (abs(dz) @ abs(wv))
    bound += r * (abs(want) + bound) + 2.0 ** -25
    assert (abs(d_x[others].double().cpu().numpy() - want) <= bound).all()
