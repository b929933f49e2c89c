"""4-bit conversion of listed rows into a result of its own: codes, scales and what
is left alone have to be equal to the byte."""
import numpy as np
import pytest
import torch

import mx4_ref
import routed_grouped_gemm_dispatch_gb300 as moe

pytestmark = pytest.mark.gpu

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("n,n_src,cols", [(1, 5, 128), (33, 40, 640), (127, 50, 256), (128, 300, 384), (129, 129, 1152),
                                          (130, 7, 2048), (300, 1000, 1408)])
def test_source_rows_alone(n, n_src, cols, dt):
    """Rows picked by a list, result row i from entry i: no status bit, and zero scales past the last row."""
    rng = np.random.default_rng(n + cols)
    x = torch.from_numpy(rng.standard_normal((n_src, cols)) * np.exp(rng.standard_normal((n_src, 1)))).to(DTYPES[dt])
    src = rng.integers(0, n_src, n).astype(np.int32)
    codes = torch.full((n + 1, cols // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-n // 128) + 1, cols // 128, 32, 4, 4), 0xEE, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.mx4_quantize(x.cuda(), src_rows=torch.from_numpy(src).cuda(), codes=codes[:n], scales=scales[:-1], status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    c, s = mx4_ref.quantize(x.double().numpy())
    assert np.array_equal(codes[:n].cpu().numpy(), mx4_ref.pack(c)[src])
    assert np.array_equal(scales[:-1].cpu().numpy(), mx4_ref.tiles(s[src]))
    assert bool((codes[n] == 0xEE).all()) and bool((scales[-1] == 0xEE).all())


def test_source_rows_alone_with_bad_entries():
    """Skipped entries leave their row, an entry past x sets the bit, and the padding is zeroed all the same."""
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((6, 256))).half()
    for src, bit in (([3, -1, 5, 0, 0], 0), ([3, 6, 5, -2, 1], moe.MOE_DEV_BAD_TABLE)):
        codes = torch.full((5, 128), 0xEE, dtype=torch.uint8, device="cuda")
        scales = torch.full((1, 2, 32, 4, 4), 0xEE, dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        moe.mx4_quantize(x.cuda(), src_rows=torch.tensor(src, dtype=torch.int32, device="cuda"), codes=codes,
                         scales=scales, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == bit
        c, s = mx4_ref.quantize(x.double().numpy())
        want_c, want_s = np.full((5, 128), 0xEE, np.uint8), np.zeros((128, 8), np.uint8)
        want_s[:5] = 0xEE
        for i, r in enumerate(src):
            if 0 <= r < 6:
                want_c[i], want_s[i] = mx4_ref.pack(c[r:r + 1])[0], s[r]
        assert np.array_equal(codes.cpu().numpy(), want_c)
        assert np.array_equal(scales.cpu().numpy(), mx4_ref.tiles(want_s))
