"""The router's losses, counts and gradients against their formulas in 64 bits.

Tolerances.  u is half a step of fp32, 2^-24, and r that of the arrays' 16-bit type.
A probability is off by at most 32u relative: expf 2 steps (4u), a sum of up to 1024 terms in a
tree of at most 32 + 5 levels of which every term passes at most 37 additions (fewer where
PER is small; positive terms, typically a few u), the reciprocal and its product 2u.
"""
import numpy as np
import pytest
import torch

import routed_grouped_gemm_dispatch_gb300 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
P_REL = 48 * U


def make(T, E, k, seqs=1, masked=False, seed=0, spread=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.randn((T, E), generator=g, device="cuda") * spread
    z -= 0.5 * torch.log(torch.arange(1, E + 1, device="cuda").float())
    s = {"z": z, "ids": torch.topk(z, k, dim=1).indices.to(torch.int32), "mask": None, "offs": None}
    if seqs > 1:
        cuts = torch.randint(0, T + 1, (seqs - 1,), generator=g, device="cuda").sort().values
        s["offs"] = torch.cat((torch.zeros_like(cuts[:1]), cuts, torch.full_like(cuts[:1], T))).to(torch.int32)
    if masked:
        s["mask"] = torch.rand((T,), generator=g, device="cuda") >= 0.3
    return s


def sequences(s):
    """Rows of each sequence that count."""
    T = s["z"].shape[0]
    b = [0, T] if s["offs"] is None else s["offs"].tolist()
    ok = np.ones(T, bool) if s["mask"] is None else s["mask"].cpu().numpy().astype(bool)
    return [np.array([t for t in range(lo, hi) if ok[t]], dtype=np.int64) for lo, hi in zip(b, b[1:])]


def softmax(z):
    """And the logsumexp; of a row of minus infinities zeros."""
    none = np.isneginf(z).all(axis=1, keepdims=True)
    top = np.where(none, 0.0, z.max(axis=1, keepdims=True))
    e = np.exp(z - top)
    total = np.where(none, 1.0, e.sum(axis=1, keepdims=True))
    return e / total, np.where(none, 0.0, top + np.log(total))[:, 0]


def finite_top(z):
    top = z.max(axis=1)
    return np.where(np.isneginf(top), 0.0, top)


def reference(s):
    """losses, counts, tokens per sequence, and the tolerances of the losses"""
    z, ids = s["z"].double().cpu().numpy(), s["ids"].cpu().numpy()
    E, k = z.shape[1], ids.shape[1]
    rows = sequences(s)
    n = sum(map(len, rows))
    bal = zl = z_tol = 0.0
    counts = np.zeros((len(rows), E), np.int64)
    for i, r in enumerate(rows):
        if not len(r):
            continue
        p, lse = softmax(z[r])
        c = ids[r].reshape(-1)
        counts[i] = np.bincount(c[(c >= 0) & (c < E)], minlength=E)
        bal += (counts[i] * p.sum(axis=0)).sum() / len(r)
        zl += (lse ** 2).sum()
        # lse: the maximum and a logarithm of a sum that is off by P_REL, each rounded
        z_tol += (2 * np.abs(lse) * (P_REL + 4 * U * (np.abs(lse) + np.abs(finite_top(z[r])) + np.log(E)))).sum() + 64 * U * (lse ** 2).sum()
    m = max(n, 1)
    losses = np.array([bal * E / (k * m), zl / m])
    # sums over a warp's tokens and a block's warps in fp32, at most 64 additions at these sizes
    return losses, counts, np.array([len(r) for r in rows] + [n]), np.array([(P_REL + 66 * U) * losses[0], z_tol / m + U * losses[1]])


SHAPES = [(1, 1, 1, 1, False), (1, 4, 2, 1, False), (2, 3, 3, 1, True), (7, 5, 1, 2, False), (31, 64, 6, 1, True),
          (32, 128, 8, 1, False), (33, 130, 8, 3, True), (64, 256, 16, 1, False), (129, 257, 4, 2, True),
          (300, 1024, 8, 5, True), (301, 1021, 16, 1, False), (1000, 60, 6, 400, True), (4097, 64, 6, 5, True),
          (9000, 255, 8, 1, True), (16384, 256, 8, 4, False), (66, 64, 6, 31, True), (5000, 48, 4, 32, True),
          (2048, 200, 8, 1, False), (1500, 1000, 8, 1, True), (700, 129, 8, 9, False), (1025, 128, 6, 3, True), (70, 96, 6, 50, True), (16, 1024, 8, 16, False)]


@pytest.mark.parametrize("T,E,k,seqs,masked", SHAPES)
def test_balance(T, E, k, seqs, masked):
    s = make(T, E, k, seqs, masked, seed=T + E)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(token_mask=s["mask"], seq_offsets=s["offs"])
    losses, counts, tokens = moe.router_balance(s["z"], s["ids"], status=status, **args)
    want, c, n, tol = reference(s)
    assert int(status) == 0
    assert np.array_equal(counts.cpu().numpy(), c) and np.array_equal(tokens.cpu().numpy(), n)
    got = losses.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol), (got, want, tol)
    # the same again, bit for bit
    again = moe.router_balance(s["z"], s["ids"], **args)
    assert all(torch.equal(a, b) for a, b in zip((losses, counts, tokens), again))


def test_balance_closed_forms():
    """Equal logits: every probability is 1/E, so the balance loss is 1 whoever is chosen, and logsumexp = log E."""
    T, E, k = 100, 48, 6
    ids = torch.stack([torch.randperm(E)[:k] for _ in range(T)]).to(torch.int32).cuda()
    losses, counts, tokens = moe.router_balance(torch.full((T, E), 0.0, device="cuda"), ids)
    want = np.array([1.0, np.log(E) ** 2])
    assert np.all(np.abs(losses.double().cpu().numpy() - want) <= 256 * U * want)
    assert int(counts.sum()) == T * k and tokens.tolist() == [T, T]


def grads_reference(s, dw, dl, counts, tokens):
    """d_z in 64 bits, and how far 32 bits may be off from it"""
    z, ids = s["z"].double().cpu().numpy(), s["ids"].cpu().numpy()
    T, E, k = z.shape[0], z.shape[1], ids.shape[1]
    dz, tol = np.zeros((T, E)), np.zeros((T, E))
    n = max(int(tokens[-1]), 1)
    for i, r in enumerate(sequences(s)):
        if not len(r):
            continue
        p, lse = softmax(z[r])
        g, mag = np.zeros((len(r), E)), np.zeros((len(r), E))
        zt = 0.0
        if dl is not None:
            g += dl[0] * E / (k * n * max(int(tokens[i]), 1)) * counts[i]
            mag += np.abs(g)
            zt = dl[1] * 2 / n * lse
        if dw is not None:
            for j in range(k):
                ok = (ids[r, j] >= 0) & (ids[r, j] < E)
                np.add.at(g, (np.arange(len(r))[ok], ids[r, j][ok]), dw[r, j][ok])
                np.add.at(mag, (np.arange(len(r))[ok], ids[r, j][ok]), np.abs(dw[r, j][ok]))
        dot = (p * g).sum(axis=1, keepdims=True)
        zt = np.reshape(zt, (-1, 1)) if np.ndim(zt) else np.full((len(r), 1), zt)
        dz[r] = p * (g - dot + zt)
        size = mag + (p * mag).sum(axis=1, keepdims=True) + np.abs(zt)
        lse_err = np.abs(zt) * (P_REL + 8 * U * (np.abs(finite_top(z[r])) + np.abs(lse) + np.log(E)))[:, None] / np.maximum(np.abs(lse), 1e-30)[:, None]
        tol[r] = p * (2 * P_REL * size + lse_err)
    return dz, tol


def check_grads(s, x, w, dw, dl, got, d_logits, counts, tokens):
    dt = x.dtype
    r = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if dt == torch.float16 else 2.0 ** -134        # half the least step
    dz, tol = grads_reference(s, None if dw is None else dw.double().cpu().numpy(),
                              None if dl is None else dl.double().cpu().numpy(), counts, tokens)
    if d_logits is not None:
        err = np.abs(d_logits.double().cpu().numpy() - dz)
        assert np.all(err <= tol + 1e-43), (err - tol).max()
    # the operand: d_z rounded once, up to 2048 tokens in two terms (each off by half a step); below 2^-27 of the
    # largest, fp16 keeps absolute steps
    dz_r = r if len(dz) > 2048 else r * r
    dz_tol = tol + (dz_r + 2 * U) * (np.abs(dz) + tol) + np.abs(dz).max(initial=0) * 2.0 ** -38 + 2.0 ** -134
    live = np.zeros(len(dz), bool)
    for rows in sequences(s):
        live[rows] = True
    dz_tol[~live] = 0
    wv, xv = w.double().cpu().numpy(), x.double().cpu().numpy()
    xv = np.where(live[:, None], xv, 0)

    def acc(k):
        return (k / 16 + 8) * 2.0 ** -23                              # fp32 sums on the tensor cores

    two = 1 if len(dz) > 2048 else 2             # terms of a sum
    for name, d, a, da, b, k in (("d_x", got[0], dz, dz_tol, wv, two * dz.shape[1]),
                                 ("d_w", got[1], dz.T, dz_tol.T, xv, two * len(dz))):
        want = a @ b
        bound = da @ np.abs(b) + acc(k) * (np.abs(a) @ np.abs(b))
        bound += r * (np.abs(want) + bound) + tiny
        err = np.abs(d.double().cpu().numpy() - want)
        assert np.isfinite(err).all() and np.all(err <= bound), (name, (err / np.maximum(bound, 1e-300)).max())


GRADS = [(1, 4, 2, 8, 1, False), (1, 64, 6, 264, 1, False), (2, 3, 3, 128, 1, True), (31, 64, 6, 256, 1, True),
         (32, 128, 8, 2048, 1, False), (65, 130, 8, 520, 3, True), (128, 256, 16, 1032, 1, False),
         (129, 257, 4, 392, 2, True), (300, 1021, 8, 768, 4, True), (1000, 60, 6, 136, 200, False),
         (2049, 64, 6, 2048, 5, True), (4097, 256, 8, 904, 1, False)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,H,seqs,masked", GRADS)
def test_backward(T, E, k, H, seqs, masked, dtype):
    s = make(T, E, k, seqs, masked, seed=T + E + H)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    w = torch.randn((E, H), generator=g, device="cuda").mul_(H ** -0.5).to(dtype)
    dw = torch.randn((T, k), generator=g, device="cuda") * 4
    dl = torch.tensor([8.0, 0.5], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(token_mask=s["mask"], seq_offsets=s["offs"], status=status)
    _, counts, tokens = moe.router_balance(s["z"], s["ids"], **kw)
    c, n = counts.cpu().numpy(), tokens.cpu().numpy()
    for a, b in ((dw, dl), (dw, None), (None, dl)):
        d_logits = torch.full((T, E), float("nan"), device="cuda")
        got = moe.router_backward(x, w, s["z"], s["ids"], a, b, counts if b is not None else None,
                                  tokens if b is not None else None, d_logits=d_logits, **kw)
        assert int(status) == 0
        check_grads(s, x, w, a, b, got, d_logits, c, n)
    again = moe.router_backward(x, w, s["z"], s["ids"], None, dl, counts, tokens, **kw)
    assert all(torch.equal(p.view(torch.int16), q.view(torch.int16)) for p, q in zip(got, again))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_what_is_masked_meets_nothing(dtype):
    """NaN and infinities in logits, ids, routed gradients and x of tokens that do not count."""
    T, E, k, H = 333, 64, 6, 264
    s = make(T, E, k, 1, True, seed=3)
    # sequences that leave tokens out at both ends and between themselves nothing
    s["offs"] = torch.tensor([5, 90, 90, 300], dtype=torch.int32, device="cuda")
    out = ~s["mask"]
    out[:5] = True
    out[300:] = True
    x, w = torch.randn((T, H), device="cuda").to(dtype), torch.randn((E, H), device="cuda").to(dtype)
    dw, dl = torch.randn((T, k), device="cuda"), torch.tensor([3.0, 0.25], device="cuda")
    kw = dict(token_mask=s["mask"], seq_offsets=s["offs"])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    clean = moe.router_balance(s["z"], s["ids"], status=status, **kw)
    clean_g = moe.router_backward(x, w, s["z"], s["ids"], dw, dl, *clean[1:], status=status, **kw)
    check_grads(s, x, w, dw, dl, clean_g, None, clean[1].cpu().numpy(), clean[2].cpu().numpy())
    for bad in (float("nan"), float("inf"), float("-inf"), 3e38):
        z, xb, dwb, ids = s["z"].clone(), x.clone(), dw.clone(), s["ids"].clone()
        z[out], xb[out], dwb[out], ids[out] = bad, bad, bad, 10 ** 6
        got = moe.router_balance(z, ids, status=status, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, clean))
        got_g = moe.router_backward(xb, w, z, ids, dwb, dl, *got[1:], status=status, **kw)
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got_g, clean_g))
        assert torch.equal(got_g[0][out], torch.zeros_like(got_g[0][out]))
    assert int(status) == 0


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min])
def test_experts_that_are_masked(low):
    """Logits of minus infinity, or of the type's lowest value: no probability, no gradient, and the others as they are."""
    T, E, k, H = 130, 72, 4, 136
    s = make(T, E, k, seed=21)
    s["z"][:, ::3] = low
    s["z"][5] = low                                      # none left, or with the lowest value one
    if low != float("-inf"):
        s["z"][5, 1] = 0.3
    s["ids"] = torch.topk(s["z"], k, dim=1).indices.to(torch.int32)
    s["ids"][5, 1:] = -1
    x, w = torch.randn((T, H), device="cuda").half(), torch.randn((E, H), device="cuda").half()
    dw, dl = torch.randn((T, k), device="cuda"), torch.tensor([1.0, 0.1], device="cuda")
    losses, counts, tokens = moe.router_balance(s["z"], s["ids"])
    want, c, n, tol = reference(s)
    assert np.array_equal(counts.cpu().numpy(), c) and np.all(np.abs(losses.double().cpu().numpy() - want) <= tol)
    d_z = torch.empty((T, E), device="cuda")
    got = moe.router_backward(x, w, s["z"], s["ids"], dw, dl, counts, tokens, d_logits=d_z)
    check_grads(s, x, w, dw, dl, got, d_z, c, n)
    assert not d_z[:, ::3].any()


def test_the_same_expert_twice():
    """A token that names an expert twice or three times: both pairs count, and both gradients."""
    T, E, k, H = 90, 20, 5, 64
    s = make(T, E, k, seed=8)
    s["ids"][:, 2] = s["ids"][:, 0]
    s["ids"][::4, 4] = s["ids"][::4, 0]
    x, w = torch.randn((T, H), device="cuda").half(), torch.randn((E, H), device="cuda").half()
    dw, dl = torch.randn((T, k), device="cuda"), torch.tensor([1.0, 0.1], device="cuda")
    losses, counts, tokens = moe.router_balance(s["z"], s["ids"])
    want, c, n, tol = reference(s)
    assert np.array_equal(counts.cpu().numpy(), c) and np.all(np.abs(losses.double().cpu().numpy() - want) <= tol)
    got = moe.router_backward(x, w, s["z"], s["ids"], dw, dl, counts, tokens)
    check_grads(s, x, w, dw, dl, got, None, c, n)
    again = moe.router_backward(x, w, s["z"], s["ids"], dw, dl, counts, tokens)
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, again))


@pytest.mark.parametrize("T", [0, 5, 200])
def test_nothing_counts(T):
    E, k, H = 40, 3, 72
    z, ids = torch.randn((T, E), device="cuda"), torch.zeros((T, k), dtype=torch.int32, device="cuda")
    x, w = torch.randn((T, H), device="cuda").half(), torch.randn((E, H), device="cuda").half()
    for kw in (dict(token_mask=torch.zeros(T, dtype=torch.bool, device="cuda")),
               dict(seq_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))) + (({},) if T == 0 else ()):
        losses, counts, tokens = moe.router_balance(z, ids, **kw)
        assert not losses.any() and not counts.any() and not tokens.any()
        d_x, d_w = torch.full_like(x, 7), torch.full_like(w, 7)
        moe.router_backward(x, w, z, ids, torch.ones((T, k), device="cuda"), torch.ones(2, device="cuda"), counts, tokens,
                            d_x=d_x, d_router_w=d_w, **kw)
        assert not d_x.any() and not d_w.any()


def test_ids_that_are_none():
    """Negative ids are skipped; ids past the last expert are skipped and reported."""
    T, E, k, H = 50, 16, 4, 64
    s = make(T, E, k, seed=9)
    s["ids"][::3, 1] = -1
    x, w = torch.randn((T, H), device="cuda").half(), torch.randn((E, H), device="cuda").half()
    dw, dl = torch.randn((T, k), device="cuda"), torch.tensor([1.0, 0.0], device="cuda")
    for bad in (False, True):
        if bad:
            s["ids"][7, 0] = E
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        losses, counts, tokens = moe.router_balance(s["z"], s["ids"], status=status)
        want, c, n, tol = reference(s)
        assert np.array_equal(counts.cpu().numpy(), c) and np.all(np.abs(losses.double().cpu().numpy() - want) <= tol)
        assert int(status) == (moe.MOE_DEV_BAD_EXPERT_ID if bad else 0)
        status.zero_()
        got = moe.router_backward(x, w, s["z"], s["ids"], dw, dl, counts, tokens, status=status)
        check_grads(s, x, w, dw, dl, got, None, c, n)
        assert int(status) == (moe.MOE_DEV_BAD_EXPERT_ID if bad else 0)


@pytest.mark.parametrize("offs", [[0, 60, 30, 100], [0, 101], [-1, 100], [0, 2 ** 31 - 1], [-2 ** 31, 50, 100]])
def test_bad_offsets_are_reported(offs):
    s = make(100, 32, 4, seed=2)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.router_balance(s["z"], s["ids"], seq_offsets=o, status=status)
    assert int(status) == moe.MOE_DEV_BAD_TABLE


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("size", [1e-30, 1e-9, 1.0, 1e6])
def test_gradients_of_any_size(size, dtype):
    """fp16 has few values below 1e-5: d_z goes into the products times a power of two, so d_x and d_W are
    right wherever their own type can hold them."""
    T, E, k, H = 256, 64, 6, 256
    s = make(T, E, k, seed=4)
    x = (torch.randn((T, H), device="cuda") * min(1.0, 1e3 / size)).to(dtype)
    w = (torch.randn((E, H), device="cuda") * min(1.0, 1e3 / size)).to(dtype)
    dw = torch.randn((T, k), device="cuda") * size
    d_logits = torch.empty((T, E), device="cuda")
    got = moe.router_backward(x, w, s["z"], s["ids"], dw, d_logits=d_logits)
    check_grads(s, x, w, dw, None, got, d_logits, None, np.array([T, T]))


def test_against_differences():
    """Gradients of the logits against differences of the loss that they belong to, in 64 bits of the formula."""
    T, E, k = 6, 10, 3
    s = make(T, E, k, 2, True, seed=12)
    dw, dl = torch.randn((T, k), device="cuda"), torch.tensor([0.7, 0.2], device="cuda")
    kw = dict(token_mask=s["mask"], seq_offsets=s["offs"])
    _, counts, tokens = moe.router_balance(s["z"], s["ids"], **kw)
    d_logits = torch.empty((T, E), device="cuda")
    x, w = torch.zeros((T, 8), device="cuda").half(), torch.zeros((E, 8), device="cuda").half()
    moe.router_backward(x, w, s["z"], s["ids"], dw, dl, counts, tokens, d_logits=d_logits, **kw)
    c, n, ids, dwn = counts.cpu().numpy(), tokens.cpu().numpy(), s["ids"].cpu().numpy(), dw.double().cpu().numpy()

    def loss(z):
        total = 0.0
        for i, r in enumerate(sequences(s)):
            if len(r):
                p, lse = softmax(z[r])
                total += 0.7 * E / (k * n[-1] * n[i]) * (c[i] * p.sum(axis=0)).sum() + 0.2 / n[-1] * (lse ** 2).sum()
                total += (np.take_along_axis(p, ids[r], axis=1) * dwn[r]).sum()
        return total

    z = s["z"].double().cpu().numpy()
    h = 1e-5
    for t in range(T):
        for e in range(E):
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            want = (loss(up) - loss(dn)) / (2 * h)
            # differences: h² of third derivatives below 10, and the losses' rounding over h
            assert abs(float(d_logits[t, e]) - want) <= 1e-9 + 1e-15 * 50 / h + 1e-5 * abs(want) + 2e-6


@pytest.mark.parametrize("T,H,E,k", [(1, 128, 1, 1), (33, 256, 5, 2), (128, 256, 64, 6), (300, 2048, 130, 8), (700, 512, 256, 16),
                                     (40000, 128, 64, 6), (20000, 256, 18, 2)])
def test_router_gives_its_logits(T, H, E, k):
    """Ids and weights are what they are without; the logits are those that the ids were chosen by."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn((T, H), generator=g, device="cuda").half()
    w = torch.randn((E, H), generator=g, device="cuda").mul_(H ** -0.5).half()
    ids, weights = moe.router_topk(x, w, k)
    guard = torch.full((T * E + 64,), 1234.0, device="cuda")
    z = guard[:T * E].view(T, E)
    ids2, weights2 = moe.router_topk(x, w, k, logits=z)
    assert torch.equal(ids, ids2) and torch.equal(weights, weights2)
    assert torch.all(guard[T * E:] == 1234.0)
    xd, wd = x.double(), w.double()
    want, size = xd @ wd.t(), xd.abs() @ wd.abs().t()
    assert torch.all((z.double() - want).abs() <= (H / 16 + 8) * 2.0 ** -23 * size + 1e-30)
    top = torch.gather(z, 1, ids.long())
    assert torch.equal(top, torch.topk(z, k, dim=1).values)
    p = torch.softmax(z.double(), dim=1).gather(1, ids.long())
    assert torch.all((weights.double() - p).abs() <= 2.0 ** -17 * p)


def test_captured_and_on_a_side_stream():
    """Balance and gradients recorded into one graph and replayed on new inputs, beside a call on another stream."""
    T, E, k, H = 700, 64, 6, 512
    a, b = make(T, E, k, 3, True, seed=1), make(T, E, k, 3, True, seed=2)
    x, w = torch.randn((T, H), device="cuda").half(), torch.randn((E, H), device="cuda").half()
    dw, dl = torch.randn((T, k), device="cuda"), torch.tensor([2.0, 0.1], device="cuda")

    def both(s):
        kw = dict(token_mask=s["mask"], seq_offsets=s["offs"])
        loss, counts, tokens = moe.router_balance(s["z"], s["ids"], **kw)
        return loss, counts, tokens, *moe.router_backward(x, w, s["z"], s["ids"], dw, dl, counts, tokens, **kw)

    want = both(b)
    both(a)
    graph = torch.cuda.CUDAGraph()
    s = {n: a[n].clone() for n in ("z", "ids", "mask", "offs")}
    with torch.cuda.graph(graph):
        got = both(s)
    for _ in range(3):
        for n in s:
            s[n].copy_(b[n])
        graph.replay()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            other = both(b)
        torch.cuda.synchronize()
        for p, q, o in zip(got, want, other):
            assert torch.equal(p, q) and torch.equal(o, q)
