"""Orthogonalised updates against the iteration in 64 bits.

Tolerances come from the iteration itself, run in 64 bits with the kernels' roundings and no others
(fp16 operands, some 15 bits of X in the a·X term, bf16 at the end): the same sizes of error enter
at the same places, though not the same errors.  Their sums over many entries agree to a few percent, so
the root mean square error may be 1.25 times the emulated one, and the largest of some 10^5 errors of
nearly normal size 2.5 times.
"""
import numpy as np
import pytest
import torch

import routed_grouped_gemm_dispatch_gb300 as moe

pytestmark = pytest.mark.gpu

ABC = (3.4445, -4.7750, 2.0315)


def r16(x, scale):
    return (x * scale).half().double() / scale


def iterate(g, steps=5, abc=ABC, eps=1e-7, rounded=False):
    """[batch, rows, cols] in 64 bits; `rounded`: with the kernels' roundings."""
    a, b, c = abc
    x = g.double()
    norm = x.flatten(1).norm(dim=1).clamp(min=eps)[:, None, None]
    tall = x.shape[1] > x.shape[2]
    x = (x.transpose(1, 2) if tall else x) / norm
    if not rounded:
        for _ in range(steps):
            A = x @ x.transpose(1, 2)
            x = a * x + (b * A + c * (A @ A)) @ x
        return x.transpose(1, 2) if tall else x
    if x.shape[1] <= 128 and x.shape[2] <= 16 * (448 if x.shape[1] <= 64 else 384):
        # on chip: a·X in 32 bits, but for the last step, which takes X as the products do; A and B in two terms
        def two(v, scale):
            hi = r16(v, scale)
            return hi + r16(v - hi, scale)

        for k in range(steps):
            hi = r16(x, 64.0)
            A = two(hi @ hi.transpose(1, 2), 1024.0)
            x = a * (hi if k + 1 == steps else x) + two(b * A + c * (A @ A), 64.0) @ hi
        return (x.transpose(1, 2) if tall else x).bfloat16().double()
    eye = torch.eye(x.shape[1], dtype=x.dtype, device=x.device)
    hi, lo = x, torch.zeros_like(x)
    if g.dtype == torch.float32:               # 16-bit inputs are exact
        hi = r16(x, 64.0)
        lo = ((x - hi) * 64 * 8192).float().to(torch.float8_e4m3fn).double() / (64 * 8192)
    for k in range(steps):
        A = hi @ hi.transpose(1, 2)
        d = A.diagonal(dim1=1, dim2=2)
        if c != 0:
            # (A + s)², s on the diagonal rounded with it, and put right on B's
            q = r16(A * (1 - eye) + torch.diag_embed(d + b / (2 * c)), 1024.0)
            B = c * (q @ q)
            s = q.diagonal(dim1=1, dim2=2) - d
            on = b * d + B.diagonal(dim1=1, dim2=2) - c * (2 * s * d + s * s)
        else:
            B, on = b * A, b * d
        B = r16(B * (1 - eye) + torch.diag_embed(on + a), 64.0)
        full = B @ hi + (a * lo if k + 1 < steps else 0)
        hi = r16(full, 64.0)
        lo = ((full - hi) * 64 * 8192).float().to(torch.float8_e4m3fn).double() / (64 * 8192)
        if k + 2 >= steps:
            lo = torch.zeros_like(lo)
    return (full.transpose(1, 2) if tall else full).bfloat16().double()


def draw(kind, batch, rows, cols, dtype, seed=0, size=1e-3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + rows + cols)

    def n(*s):
        return torch.randn(s, generator=g, device="cuda")

    r = min(rows, cols)
    x = {"normal": lambda: n(batch, rows, cols),
         "low rank": lambda: n(batch, rows, max(1, r // 8)) @ n(batch, max(1, r // 8), cols) + 0.01 * n(batch, rows, cols),
         "rank one": lambda: n(batch, rows, 1) @ n(batch, 1, cols),
         "rows of zeros": lambda: n(batch, rows, cols) * (torch.arange(rows, device="cuda") % 3 > 0)[:, None]}[kind]()
    return (x * size).to(dtype)


def check(update, got, **kw):
    u = update if update.dim() == 3 else update[None]
    o = (got if got.dim() == 3 else got[None]).double()
    want, sim = iterate(u, **kw), iterate(u, rounded=True, **kw)
    assert got.dtype == torch.bfloat16 and got.shape == update.shape
    for i in range(len(u)):
        err, ref = o[i] - want[i], sim[i] - want[i]
        rms = float(want[i].square().mean().sqrt())
        assert float(err.square().mean().sqrt()) <= 1.25 * float(ref.square().mean().sqrt()) + 1e-9 * rms
        assert float(err.abs().max()) <= 2.5 * float(ref.abs().max()) + 1e-9 * rms


# sizes around the tiles' (128, 256), of whole and broken 16-byte rows, wide, square and tall
SIZES = [(1, 64, 96), (1, 64, 2048), (2, 128, 128), (1, 129, 130), (3, 333, 1001), (1, 256, 256), (2, 257, 300), (1, 500, 200),
         (1, 1001, 77), (2, 520, 264), (5, 96, 640), (1, 600, 1544), (1, 1408, 768), (1, 100, 6144), (2, 6100, 128), (1, 90, 6150), (40, 65, 129), (1, 64, 7168), (1, 7100, 40),
         (2, 40, 7200),
         (200, 16, 40), (20, 128, 520)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,rows,cols", SIZES)
def test_sizes(batch, rows, cols, dtype):
    u = draw("normal", batch, rows, cols, dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(u, moe.orthogonalize(u, status=status))
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["low rank", "rank one", "rows of zeros"])
@pytest.mark.parametrize("rows,cols", [(200, 520), (700, 300), (256, 1024), (64, 300), (2048, 100)])
def test_spectra(kind, rows, cols, dtype):
    u = draw(kind, 2, rows, cols, dtype)
    check(u, moe.orthogonalize(u))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 9), (5, 1), (2, 3), (8, 8), (17, 5), (40, 33)])
def test_tiny(rows, cols):
    """Few entries: each is held against the emulated error's size, the type's rounding and the operands'."""
    u = draw("normal", 4, rows, cols, torch.float32)
    got, want = moe.orthogonalize(u).double(), iterate(u)
    # one rounding of the result, 2^-8 of it, and five steps of operands of 11 bits: each moves X by at most
    # (|b| + |c|·2)·1.2³·4·2^-11 ≤ 3.1e-2 of the largest singular value, 1.2, where errors add up without
    # cancelling; the map contracts what came before (|slope| <= 1.2 from the second step at these sizes)
    assert float((got - want).abs().max()) <= 2.0 ** -8 * 1.3 + 3.1e-2 * 1.2


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_either_side_and_each_by_itself(dtype):
    """A stack gives what its matrices give alone, bit for bit, and a power of two changes nothing (where the type
    holds the product exactly: fp16 does not below 2^-14).  The transpose gives the transpose, up
    to the order in which its squares are summed."""
    u = draw("normal", 3, 264, 400, dtype, size=0.25)
    y = moe.orthogonalize(u)
    t = u.transpose(1, 2).contiguous()
    check(t, moe.orthogonalize(t))
    for i in range(3):
        assert torch.equal(moe.orthogonalize(u[i]), y[i])
        v = u[i] * 0.125
        exact = torch.equal(v.float() * 8, u[i].float())
        assert exact or dtype == torch.float16
        if exact:
            assert torch.equal(moe.orthogonalize(v), y[i])
    assert torch.equal(moe.orthogonalize(u), y)


def test_zeros_and_what_is_not_finite():
    """A matrix of zeros stays zeros, one with a NaN or an infinity becomes NaN, and the others are what they are."""
    u = draw("normal", 6, 130, 200, torch.float32)
    y = moe.orthogonalize(u)
    v = u.clone()
    v[1] = 0
    v[2, 5, 7] = float("nan")
    v[4, 129, 199] = float("-inf")
    v[5] *= 1e25                                     # its squares leave fp32
    z = moe.orthogonalize(v)
    for i in (0, 3):
        assert torch.equal(z[i], y[i])
    assert not z[1].any()
    for i in (2, 4, 5):
        assert torch.isnan(z[i]).all()


def test_eps():
    """Below eps the update is divided by eps: it stays small instead of becoming a direction of noise."""
    u = draw("normal", 1, 64, 64, torch.float32, size=1e-9)
    check(u, moe.orthogonalize(u, eps=1e-3), eps=1e-3)
    check(u, moe.orthogonalize(u, eps=0.0), eps=0.0)


@pytest.mark.parametrize("steps,abc", [(1, ABC), (2, ABC), (3, (1.5, -0.5, 0.0)), (12, (2.0, -1.5, 0.5)), (6, ABC)])
def test_steps_and_coefficients(steps, abc):
    for dt in (torch.float32, torch.bfloat16):
        u = draw("normal", 1, 130, 300, dt)
        check(u, moe.orthogonalize(u, steps=steps, coefficients=abc), steps=steps, abc=abc)


def test_given_out_workspace_and_guards():
    """Everything written lies in `out` and the workspace that were given."""
    for rows, cols in ((77, 130), (131, 64)):
        u = draw("normal", 2, rows, cols, torch.bfloat16)
        n = moe.orthogonalize_workspace_bytes(2, rows, cols)
        ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        buf = torch.full((2 * rows * cols + 2048,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[:2 * rows * cols].view(2, rows, cols)
        got = moe.orthogonalize(u, out=out, workspace=ws[:n])
        assert got.data_ptr() == out.data_ptr()
        assert torch.all(ws[n:] == 0x5A) and torch.all(buf[2 * rows * cols:] == 7.0)
        assert torch.equal(out, moe.orthogonalize(u))
    assert moe.orthogonalize(torch.empty((0, 8, 8), device="cuda")).shape == (0, 8, 8)


def test_captured_and_on_two_streams():
    a, b = draw("normal", 2, 200, 300, torch.bfloat16, 1), draw("normal", 2, 200, 300, torch.bfloat16, 2)
    want = moe.orthogonalize(b)
    u = a.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = moe.orthogonalize(u)
    side = torch.cuda.Stream()
    for _ in range(3):
        u.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        other = moe.orthogonalize(b, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(other, want)


def test_large_calls_at_once():
    """Two calls that each fill the device, on two streams: tiles go to whatever pairs run."""
    a, b = draw("normal", 4, 600, 1544, torch.bfloat16, 1), draw("normal", 1, 1408, 768, torch.float32, 2)
    c = draw("normal", 8, 100, 900, torch.float16, 3)
    want = [moe.orthogonalize(v) for v in (a, b, c)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        got = [moe.orthogonalize(v, stream=s) for v, s in zip((a, b, c), streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_past_31_bits():
    """A stack of more than 2^31 elements: the last matrix is what it is alone."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    u = torch.zeros((1100, 1024, 2048), dtype=torch.bfloat16, device="cuda")
    last = draw("normal", 1, 1024, 2048, torch.bfloat16, 4)
    u[-1], u[7] = last[0], last[0]
    y = moe.orthogonalize(u, steps=2)
    alone = moe.orthogonalize(last, steps=2)[0]
    assert torch.equal(y[-1], alone) and torch.equal(y[7], alone)
    assert not y[6].any() and not y[-2].any()
