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
