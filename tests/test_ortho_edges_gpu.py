"""Orthogonalised updates where clusters start unevenly, at norms and sizes that the other tests leave out; against the
iteration in 64 bits, with the tolerances of test_ortho_gpu."""
import pytest
import torch

import routed_grouped_gemm_dispatch_gb300 as moe
import test_ortho_gpu as ortho

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 2048), (4, 2, 1100), (9, 2048, 8), (60, 16, 130)])
def test_blocks_that_start_apart(batch, rows, cols):
    """One norm over all blocks of a cluster, whenever each of them starts: next to no work before they exchange their
    parts, on a device that another stream keeps busy, always the same result."""
    u = ortho.draw("normal", batch, rows, cols, torch.float32)
    want = moe.orthogonalize(u)
    ortho.check(u, want)
    side, busy = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(side):
            busy = busy.sin()
        got.append(moe.orthogonalize(u))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


TINY = 2.0 ** -69                # a root mean square below which fp32's squares no longer give the norm


@pytest.mark.parametrize("eps", [0.0, 1e-45, torch.finfo(torch.float32).tiny, 2.0 ** -122, 1e-30, 1e-7])
@pytest.mark.parametrize("rows,cols", [(64, 96), (130, 200), (400, 150)])
def test_zeros_whatever_eps(rows, cols, eps):
    """A matrix of zeros stays zeros however small eps is, and its neighbour is what it is."""
    for dt in (torch.float32, torch.bfloat16):
        u = ortho.draw("normal", 2, rows, cols, dt)
        want = moe.orthogonalize(u)
        u[0] = 0
        got = moe.orthogonalize(u, eps=eps)
        assert not got[0].any() and torch.equal(got[1], want[1])


@pytest.mark.parametrize("size", [1e-19, 1e-20, 5e-22, 3e-23])
@pytest.mark.parametrize("rows,cols", [(64, 96), (130, 200), (400, 150)])
def test_values_whose_squares_leave_fp32(rows, cols, size):
    """The norm is no less than that of entries of 2^-69, so nothing is divided by a norm that fp32 lost.  Squares of
    2^-138 are off by 2^-12 of themselves at most (fp32 has steps of 2^-149), which moves the norm and the first X by half of
    that: below the roundings that the tolerance already counts."""
    u = ortho.draw("normal", 2, rows, cols, torch.float32, size=size)
    ortho.check(u, moe.orthogonalize(u, eps=0.0), eps=TINY * (rows * cols) ** 0.5)


# By the widths that the tiles of A and of X get: narrow and wide, wide and narrow, both wide (both narrow: most of
# test_ortho_gpu), with whole and ragged panels, wide and tall
WIDTHS = [(5, 130, 7170), (3, 5000, 257), (16, 256, 1704), (16, 513, 520), (24, 520, 513), (16, 513, 700), (16, 701, 513),
          (40, 400, 520), (8, 1001, 900), (9, 1024, 768)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["normal", "low rank"])
@pytest.mark.parametrize("batch,rows,cols", WIDTHS)
def test_tiles_of_every_width(batch, rows, cols, kind, dtype):
    u = ortho.draw(kind, batch, rows, cols, dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # (a workspace of NaN: nothing of it is read before it is written)
    ws = torch.full((moe.orthogonalize_workspace_bytes(batch, rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    got = moe.orthogonalize(u, workspace=ws, status=status)
    ortho.check(u, got)
    assert int(status) == 0 and torch.equal(got, moe.orthogonalize(u))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 9), (5, 1), (2, 3), (8, 8), (17, 5), (40, 33)])
def test_many_tiny_matrices(rows, cols):
    """Matrices with few entries, enough of them for their errors' root mean square to be that of the emulation: the same
    bound as for large ones, over all."""
    u = ortho.draw("normal", 4000 // min(rows, cols) + 100, rows, cols, torch.float32)
    got, want, sim = moe.orthogonalize(u).double(), ortho.iterate(u), ortho.iterate(u, rounded=True)
    err, ref = got - want, sim - want
    assert float(err.square().mean().sqrt()) <= 1.25 * float(ref.square().mean().sqrt())
    assert float(err.abs().max()) <= 2.5 * float(ref.abs().max())


def test_the_largest_matrix():
    """65536 x 65536, more than 2^32 elements: a diagonal of ±1 in some order stays one, and its values follow the polynomial of
    one number.  (Every sum has a single term: X, A and B are rounded to 11 bits in each step and the result to bf16.)"""
    n = 65536
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    at = torch.randperm(n, generator=g, device="cuda")
    sign = torch.randint(0, 2, (n,), generator=g, device="cuda").mul_(2).sub_(1).bfloat16()
    u = torch.zeros((n, n), dtype=torch.bfloat16, device="cuda")
    u[torch.arange(n, device="cuda"), at] = sign
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = moe.orthogonalize(u, steps=2, status=status)
    assert int(status) == 0
    x, (a, b, c) = 1 / 256, ortho.ABC
    for _ in range(2):
        x = a * x + b * x ** 3 + c * x ** 5
    got = y[torch.arange(n, device="cuda"), at] * sign
    # two steps whose B (a on its diagonal, 3.4) and X are off by 2^-12 each, then bf16's 2^-8 at most
    assert float((got.double() / x - 1).abs().max()) <= 2.0 ** -8 + 6 * 2.0 ** -12
    y[torch.arange(n, device="cuda"), at] = 0
    assert not any(bool(part.any()) for part in y.split(4096))


@pytest.mark.parametrize("rows,cols,steps", [(2, 2, 5), (129, 130, 2)])
def test_the_most_matrices(rows, cols, steps):
    n = 65535
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    u = torch.randn((n, rows, cols), generator=g, device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = moe.orthogonalize(u, steps=steps, status=status)
    assert int(status) == 0 and y.shape == u.shape
    for part in (slice(0, 50), slice(n // 2, n // 2 + 50), slice(n - 50, n)):
        want, sim = ortho.iterate(u[part], steps=steps), ortho.iterate(u[part], steps=steps, rounded=True)
        err, ref = y[part].double() - want, sim - want
        assert float(err.square().mean().sqrt()) <= 1.25 * float(ref.square().mean().sqrt())
        assert float(err.abs().max()) <= 2.5 * float(ref.abs().max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("share", [1e-2, 1e-4, 1e-6])
@pytest.mark.parametrize("rows,cols", [(64, 512), (200, 520), (1000, 600)])
def test_norms_far_below_eps(rows, cols, share, dtype):
    """Where eps is much more than the norm, fp16 holds X times 2^6 in steps of 2^-24, uniformly off by 2^-25/√3 at root mean
    square: 2.7e-10 of X, in the first one up to twice that (what is left of 1/eps beside a power of two is below 2).  The products
    do not matter there, so a step multiplies by a = 3.4445: errors of five X add up to 2.7e-10·√((2a⁵)² + a⁸ + a⁶ + a⁴ + a²)
    = 2.7e-7, and the result's own rounding is as ever."""
    u = ortho.draw("normal", 2, rows, cols, dtype)
    eps = float(u[0].float().norm()) / share
    got, want = moe.orthogonalize(u, eps=eps), ortho.iterate(u, eps=eps)
    err = (got.double() - want).square().mean().sqrt()
    assert float(err) <= 2.5e-3 * float(want.square().mean().sqrt()) + 2.8e-7
