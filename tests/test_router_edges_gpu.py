"""The router's losses and gradients where neighbouring tokens share experts, with peaked logits, and at sizes and tables
that the other tests leave out; against the formulas in 64 bits, with the tolerances of test_router_train_gpu unless
a test derives its own."""
import numpy as np
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


U = router.U


def peaked_reference(s, dw, dl):
    """Losses and d_z in 64 bits, and how far 32 bits may be off, for logits at any distance from their row's maximum.

    An exponential is 2^((z − top)·log2 e): the difference, the constant and the product are rounded by u each, so at a distance D
    it is off by 3u·D of itself, ex2 by 4u more, and it may be 2^-126 less (results below are flushed to zero).  The sum
    adds its terms' errors and at most 37 additions, u each; the reciprocal and the product take 3u.  So a probability is off by
    (3D + 3·Σ p·D + 48)·u of itself, and the logarithm of the sum by (3·Σ p·D + 41)·u."""
    z, ids = s["z"].double().cpu().numpy(), s["ids"].cpu().numpy()
    (T, E), k = z.shape, ids.shape[1]
    rows = router.sequences(s)
    n = max(sum(map(len, rows)), 1)
    bal = zl = bal_tol = zl_tol = 0.0
    dz, tol = np.zeros((T, E)), np.zeros((T, E))
    for r in rows:
        if not len(r):
            continue
        p, lse = router.softmax(z[r])
        top = z[r].max(axis=1)
        D = top[:, None] - z[r]
        mean_D = (p * D).sum(axis=1, keepdims=True)
        p_tol = p * (3 * D + 3 * mean_D + 48) * U + 2.0 ** -125
        lse_tol = ((3 * mean_D[:, 0] + 41) + 2 * np.abs(lse - top) + np.abs(lse)) * U
        counts = np.bincount(ids[r].reshape(-1), minlength=E)
        # sums over tokens: at most 64 additions in fp32, pairs of fp32 beyond
        bal += (counts * p.sum(axis=0)).sum() / len(r)
        bal_tol += (counts * (p_tol + 68 * U * p).sum(axis=0)).sum() / len(r)
        zl += (lse ** 2).sum()
        zl_tol += (2 * np.abs(lse) * lse_tol + 68 * U * lse ** 2).sum()
        g, mag = np.zeros((len(r), E)), np.zeros((len(r), E))
        g += dl[0] * E / (k * n * len(r)) * counts
        mag += np.abs(g)
        for j in range(k):
            np.add.at(g, (np.arange(len(r)), ids[r, j]), dw[r, j])
            np.add.at(mag, (np.arange(len(r)), ids[r, j]), np.abs(dw[r, j]))
        zt = (dl[1] * 2 / n * lse)[:, None]
        zt_tol = (np.abs(dl[1]) * 2 / n * lse_tol)[:, None] + 4 * U * np.abs(zt)
        dot = (p * g).sum(axis=1, keepdims=True)
        # g by a few operations; its product with p summed over at most 37 additions
        dot_tol = ((p_tol + 48 * U * p) * mag).sum(axis=1, keepdims=True)
        dz[r] = p * (g - dot + zt)
        size = mag + (p * mag).sum(axis=1, keepdims=True) + np.abs(zt)
        tol[r] = p_tol * size + p * (dot_tol + zt_tol + 16 * U * size)
    return (np.array([bal * E / (k * n), zl / n]), np.array([bal_tol * E / (k * n), zl_tol / n]) * (1 + 16 * U), dz, tol)


@pytest.mark.parametrize("spread", [3.0, 10.0, 30.0])
@pytest.mark.parametrize("T,E,k,seqs,masked", [(300, 64, 6, 1, False), (5000, 128, 8, 5, True), (700, 130, 4, 1, False),
                                               (30000, 60, 6, 3, True), (2500, 1000, 8, 40, False)])
def test_peaked_logits(T, E, k, seqs, masked, spread):
    """A router that is sure: most experts' probabilities are tiny or zero."""
    s = router.make(T, E, k, seqs, masked, seed=T + int(spread), spread=spread)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x, w = torch.zeros((T, 8), device="cuda").half(), torch.zeros((E, 8), device="cuda").half()
    dw, dl = torch.randn((T, k), generator=g, device="cuda"), torch.tensor([8.0, 0.5], device="cuda")
    kw = dict(token_mask=s["mask"], seq_offsets=s["offs"])
    losses, counts, tokens = moe.router_balance(s["z"], s["ids"], **kw)
    want, tol, dz, dz_tol = peaked_reference(s, dw.double().cpu().numpy(), dl.double().cpu().numpy())
    assert (abs(losses.double().cpu().numpy() - want) <= tol).all()
    d_logits = torch.empty((T, E), device="cuda")
    moe.router_backward(x, w, s["z"], s["ids"], dw, dl, counts, tokens, d_logits=d_logits, **kw)
    assert (abs(d_logits.double().cpu().numpy() - dz) <= dz_tol + 1e-43).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_what_is_left_out_of_many_tokens(dtype):
    """Sequences that leave tokens out at both ends, a mask, and NaN in all of those: the losses in two launches, and d_W in
    parts, as they are without."""
    T, E, k, H = 20000, 64, 6, 264
    s = router.make(T, E, k, 1, True, seed=3)
    s["offs"] = torch.tensor([5, 9000, 9000, 19000], dtype=torch.int32, device="cuda")
    out = ~s["mask"]
    out[:5] = True
    out[19000:] = True
    x, w = torch.randn((T, H), device="cuda").to(dtype), torch.randn((E, H), device="cuda").to(dtype)
    dw, dl = torch.randn((T, k), device="cuda"), torch.tensor([3.0, 0.25], device="cuda")
    kw = dict(token_mask=s["mask"], seq_offsets=s["offs"])
    clean = moe.router_balance(s["z"], s["ids"], **kw)
    want, c, n, tol = router.reference(s)
    assert (abs(clean[0].double().cpu().numpy() - want) <= tol).all()
    assert (clean[1].cpu().numpy() == c).all() and (clean[2].cpu().numpy() == n).all()
    clean_g = moe.router_backward(x, w, s["z"], s["ids"], dw, dl, *clean[1:], **kw)
    router.check_grads(s, x, w, dw, dl, clean_g, None, c, n)
    z, xb, dwb, ids = s["z"].clone(), x.clone(), dw.clone(), s["ids"].clone()
    z[out], xb[out], dwb[out], ids[out] = float("nan"), float("nan"), float("nan"), 10 ** 6
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = moe.router_balance(z, ids, status=status, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, clean))
    got_g = moe.router_backward(xb, w, z, ids, dwb, dl, *got[1:], status=status, **kw)
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got_g, clean_g))
    assert not got_g[0][out].any() and int(status) == 0


def test_the_most_tokens():
    """2^24 of them: losses, counts and gradients against 64 bits, on the device."""
    T, E, k, H = 1 << 24, 5, 2, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(24)
    z = torch.randn((T, E), generator=g, device="cuda")
    ids = torch.topk(z, k, dim=1).indices.to(torch.int32)
    mask = torch.rand((T,), generator=g, device="cuda") >= 0.25
    x, w = torch.randn((T, H), generator=g, device="cuda").half(), torch.randn((E, H), generator=g, device="cuda").half()
    dw, dl = torch.randn((T, k), generator=g, device="cuda"), torch.tensor([2.0 ** 24, 2.0 ** 22], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    losses, counts, tokens = moe.router_balance(z, ids, token_mask=mask, status=status)
    d_z = torch.empty((T, E), device="cuda")
    d_x, d_w = moe.router_backward(x, w, z, ids, dw, dl, counts, tokens, token_mask=mask, d_logits=d_z, status=status)
    assert int(status) == 0
    live = mask.double()[:, None]
    n = int(mask.sum())
    assert tokens.tolist() == [n, n]
    assert torch.equal(counts[0].long(), torch.bincount(ids[mask].reshape(-1).long(), minlength=E))
    zd = z.double()
    p, lse = torch.softmax(zd, dim=1), torch.logsumexp(zd, dim=1)
    f, P = counts[0].double(), (p * live).sum(dim=0)
    want = torch.stack(((f * P).sum() / n * E / (k * n), (lse.square() * live[:, 0]).sum() / n))
    # a block has 2^24 / 304 tokens, of which a lane adds every 32nd in fp32, then lanes, warps and blocks
    assert bool(((losses.double() - want).abs() <= (router.P_REL + (55200 / 32 + 70) * U) * 2 * want).all())
    share = float(dl[0]) * E / (k * n * n) * f
    gz = share + torch.zeros_like(p).scatter_add_(1, ids.long(), dw.double())
    zt = (float(dl[1]) * 2 / n * lse)[:, None]
    ref = p * (gz - (p * gz).sum(dim=1, keepdim=True) + zt) * live
    mag = gz.abs() + share
    size = mag + (p * mag).sum(dim=1, keepdim=True) + zt.abs() + float(dl[1]) * 2 / n
    tol = p * 2 * router.P_REL * size * live
    assert bool(((d_z.double() - ref).abs() <= tol).all())
    r = 2.0 ** -11
    tol = tol + (r + 2 * U) * (ref.abs() + tol) + ref.abs().max() * 2.0 ** -38 * live
    for got, a, da, b, terms in ((d_x, ref, tol, w.double(), E), (d_w, ref.t(), tol.t(), x.double(), T)):
        want = a @ b
        bound = da @ b.abs() + (terms / 16 + 8) * 2.0 ** -23 * (a.abs() @ b.abs())
        bound += r * (want.abs() + bound) + 2.0 ** -25
        assert bool(((got.double() - want).abs() <= bound).all())


def test_the_most_sequences():
    T, E, k, S, H = 150000, 40, 3, 65535, 16
    s = router.make(T, E, k, S, True, seed=5)
    losses, counts, tokens = moe.router_balance(s["z"], s["ids"], token_mask=s["mask"], seq_offsets=s["offs"])
    want, c, n, tol = router.reference(s)
    assert (counts.cpu().numpy() == c).all() and (tokens.cpu().numpy() == n).all()
    assert (abs(losses.double().cpu().numpy() - want) <= tol).all()
    x, w = torch.randn((T, H), device="cuda").half(), torch.randn((E, H), device="cuda").half()
    dw, dl = torch.randn((T, k), device="cuda"), torch.tensor([3e5, 1e4], device="cuda")
    d_logits = torch.empty((T, E), device="cuda")
    got = moe.router_backward(x, w, s["z"], s["ids"], dw, dl, counts, tokens, token_mask=s["mask"], seq_offsets=s["offs"],
                              d_logits=d_logits)
    router.check_grads(s, x, w, dw, dl, got, d_logits, c, n)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_the_widest_tokens(dtype):
    T, E, k, H = 3, 3, 2, 1 << 20
    s = router.make(T, E, k, seed=6)
    x, w = torch.randn((T, H), device="cuda").to(dtype), torch.randn((E, H), device="cuda").to(dtype)
    dw = torch.randn((T, k), device="cuda")
    got = moe.router_backward(x, w, s["z"], s["ids"], dw)
    router.check_grads(s, x, w, dw, None, got, None, None, [T, T])
