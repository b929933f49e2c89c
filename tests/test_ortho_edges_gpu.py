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
