"""4-bit conversion of listed rows into a result of its own, and tables that point outside
their arrays in both grouped forms and on both kernels: what is written and what is left
alone have to be equal to the byte."""
import numpy as np
import pytest
import torch

import mx4_ref
import routed_grouped_gemm_dispatch_gb300 as moe
from gpu_side import sentinel
from moe_cases import SENTINEL

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


def operand(rng, rows, cols):
    c, s = mx4_ref.quantize(rng.standard_normal((rows, cols)))
    return torch.from_numpy(mx4_ref.pack(c)).cuda(), torch.from_numpy(mx4_ref.tiles(s)).cuda()


@pytest.mark.parametrize("form", ["gate_up", "down"])
@pytest.mark.parametrize("T,top_k,E", [(5, 2, 8), (100, 2, 8), (300, 2, 4)], ids=["few rows", "few rows, two blocks", "pairs"])
def test_bad_tables(T, top_k, E, form):
    """An entry that points outside its array leaves its block out, sets the bit and changes no other block."""
    rng = np.random.default_rng(T)
    k, n = 256, 384
    ids = torch.from_numpy(np.argsort(rng.random((T, E)), axis=1)[:, :top_k].astype(np.int32).copy()).cuda()
    t = moe.build_dispatch(ids, E)
    rows = t["group_idx_for_bx"].numel() * 128
    a, sa = operand(rng, rows, k)
    b, sb = operand(rng, E * n, k)
    b2, sb2 = operand(rng, E * n, k)
    w = torch.from_numpy(rng.random(T * top_k).astype(np.float32)).cuda()
    names = ("group_sizes", "group_offsets", "group_padded_offsets", "group_idx_for_bx")

    def run(tab, status=None):
        out = sentinel(rows, n)
        if form == "down":
            moe.mx4_down(a, sa, b.view(E, n, -1), sb, w, *(tab[x] for x in names), out, status=status)
        else:
            moe.mx4_gate_up(a, sa, b.view(E, n, -1), sb, b2.view(E, n, -1), sb2, tab[names[0]], tab[names[2]],
                            tab[names[3]], out, status=status)
        torch.cuda.synchronize()
        return out.view(torch.int16)

    want = run(t)
    assert int(t["group_sizes"][0]) > 0 and not bool((want[0] == SENTINEL).all())
    # where expert 0's rows end
    after = int(t["group_padded_offsets"][1])
    cases = [("group_idx_for_bx", E, 128), ("group_idx_for_bx", -1, 128), ("group_idx_for_bx", 1 << 30, 128),
             ("group_padded_offsets", 128, after)]
    if form == "down":
        cases += [("group_offsets", 1 << 20, after), ("group_offsets", -T * top_k - 5, after)]
    for name, value, first in cases:
        bad = {x: v.clone() for x, v in t.items()}
        bad[name][0] = value
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run(bad, status)
        assert int(status.item()) == moe.MOE_DEV_BAD_TABLE, (name, value)
        assert bool((got[:128] == SENTINEL).all()), (name, value)
        assert torch.equal(got[first:], want[first:]), (name, value)
