"""4-bit conversion and products against their definition.

Codes, scales and the values read back have to be equal.  A product is exact in
its terms; its fp32 sum over k is off by at most 2^-23 of the sum of absolute
terms per addition, k/16 + 4 of them (as for 16-bit operands), and the result is
rounded once to 16 bits (half a step, and half of fp16's smallest subnormal).
"""
import numpy as np
import pytest
import torch

import mx4_ref
import routed_grouped_gemm_dispatch_gb300 as moe
from gpu_side import sentinel
from moe_cases import SENTINEL

pytestmark = pytest.mark.gpu

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
OUT = [torch.float16, torch.bfloat16]


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    return 2.0 ** -25 if dt == torch.float16 else 0.0


def acc(k):
    return (k / 16 + 4) * 2.0 ** -23


def special_rows(cols, dt, rng):
    """Rows that exercise the edges of the conversion, in type dt."""
    info = torch.finfo(dt)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.0, 4.0, 0.0, 0.5, 7.9])
    rows = [np.zeros(cols), np.full(cols, -0.0)]
    for scale in (1.0, 2.0 ** -9, 2.0 ** 7):
        rows.append(np.resize(ties * scale, cols) * np.where(rng.random(cols) < 0.5, -1, 1))
    rows.append(np.full(cols, info.max))
    rows.append(-np.full(cols, info.max) * rng.random(cols))
    rows.append(np.full(cols, info.tiny) * rng.random(cols))                        # around the normal limit
    rows.append(np.full(cols, info.smallest_normal * info.eps) * rng.integers(0, 9, cols))   # subnormal
    one_bad = rng.standard_normal(cols)
    one_bad[5], one_bad[40], one_bad[77], one_bad[100] = np.inf, -np.inf, np.nan, info.max
    rows.append(one_bad)
    rows.append(np.where(np.arange(cols) % 32 == 31, 1.0, 0.0))                      # the maximum in the last lane
    rows.append(np.ldexp(1.0, -(np.arange(cols) % 32)))
    return torch.from_numpy(np.stack(rows)).to(dt)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 256), (31, 384), (33, 1152), (127, 1024), (128, 1280), (129, 2048),
                                       (300, 1408), (700, 128)])
def test_quantize_and_back(rows, cols, dt):
    rng = np.random.default_rng(rows * 7 + cols)
    t = DTYPES[dt]
    x = torch.from_numpy(rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)) * 3)).to(t)
    sp = special_rows(cols, t, rng)
    x[:min(rows, len(sp))] = sp[:rows]
    codes = torch.full((rows, cols // 2), 0xEE, dtype=torch.uint8, device="cuda")
    buf = torch.full((-(-rows // 128) + 1, cols // 128, 32, 4, 4), 0xEE, dtype=torch.uint8, device="cuda")
    moe.mx4_quantize(x.cuda(), codes=codes, scales=buf[:-1])
    c, s = mx4_ref.quantize(x.double().numpy())
    torch.cuda.synchronize()
    assert np.array_equal(codes.cpu().numpy(), mx4_ref.pack(c))
    assert np.array_equal(buf[:-1].cpu().numpy(), mx4_ref.tiles(s))         # zeros past the last row
    assert bool((buf[-1] == 0xEE).all())
    want = torch.from_numpy(mx4_ref.values(c, s))
    for o in DTYPES.values():
        got = moe.mx4_dequantize(codes, buf[:-1], o).cpu()
        # one rounding from the exact value (fp32 first where it is exact: every value is)
        assert torch.equal(got.nan_to_num(nan=123.0), want.float().to(o).nan_to_num(nan=123.0))


def test_every_code_and_scale_reads_back():
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 8))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, axis=1)
    got = moe.mx4_dequantize(torch.from_numpy(mx4_ref.pack(codes)).cuda(), torch.from_numpy(mx4_ref.tiles(scales)).cuda(),
                             torch.float32).cpu().numpy().astype(np.float64)
    want = mx4_ref.values(codes, scales)
    # 4·2^126 and 6·2^126 and above are past fp32's range
    with np.errstate(over="ignore"):
        want = want.astype(np.float32).astype(np.float64)
    assert np.array_equal(np.nan_to_num(got, nan=1.25), np.nan_to_num(want, nan=1.25))


def test_weight_stack_is_its_rows():
    x = torch.randn((3, 256, 384), device="cuda").half()
    c3, s3 = moe.mx4_quantize(x)
    c2, s2 = moe.mx4_quantize(x.view(768, 384))
    assert c3.shape == (3, 256, 192) and torch.equal(c3.view(768, 192), c2) and torch.equal(s3, s2)


@pytest.mark.parametrize("copies", [1, 3, 8])
def test_row_lists(copies):
    rng = np.random.default_rng(copies)
    n_src, n_dest, cols, n = 40, 400, 640, 30
    x = torch.from_numpy(rng.standard_normal((n_src, cols))).half()
    src = rng.integers(0, n_src, n).astype(np.int32)
    dest = rng.permutation(n_dest)[:n * copies].reshape(n, copies).astype(np.int32)
    src[4] = -1                                  # skipped
    dest[6, 0] = -1
    src[9], dest[11, copies - 1] = n_src, n_dest  # out of range: skipped and reported
    codes = torch.full((n_dest, cols // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((4, cols // 128, 32, 4, 4), 0xEE, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.mx4_quantize(x.cuda(), src_rows=torch.from_numpy(src).cuda(), dest_rows=torch.from_numpy(dest).cuda(), codes=codes,
                     scales=scales, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == moe.MOE_DEV_BAD_TABLE
    c, s = mx4_ref.quantize(x.double().numpy())
    want_c = np.full((n_dest, cols // 2), 0xEE, np.uint8)
    want_s = np.full((512, cols // 32), 0xEE, np.uint8)
    for i in range(n):
        for d in dest[i]:
            if 0 <= src[i] < n_src and 0 <= d < n_dest:
                want_c[d], want_s[d] = mx4_ref.pack(c[src[i]][None])[0], s[src[i]]
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(scales.cpu().numpy(), mx4_ref.tiles(want_s))


def random_operand(rng, rows, cols, spread=0.0, std=1.0):
    """Codes, tiled scales (device) and fp64 values of a random 4-bit array."""
    x = rng.standard_normal((rows, cols)) * std * np.exp2(np.round(rng.standard_normal((rows, 1)) * spread))
    c, s = mx4_ref.quantize(x)
    return (torch.from_numpy(mx4_ref.pack(c)).cuda(), torch.from_numpy(mx4_ref.tiles(s)).cuda(),
            torch.from_numpy(mx4_ref.values(c, s)).cuda())


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - tol).max()):.3e}"


@pytest.mark.parametrize("dt", OUT, ids=["fp16", "bf16"])
@pytest.mark.parametrize("rows,k,n", [(1, 128, 128), (2, 256, 256), (3, 384, 384), (31, 640, 128), (33, 128, 640),
                                      (127, 256, 1152), (128, 1408, 256), (129, 2048, 384), (257, 896, 512),
                                      (300, 256, 2048), (1111, 512, 640), (17, 256, 128), (48, 128, 128),
                                      (64, 1152, 256), (65, 256, 384), (4500, 256, 384)])
def test_matmul(rows, k, n, dt):
    rng = np.random.default_rng(rows + k + n)
    a, sa, va = random_operand(rng, rows, k, spread=1.0)
    b, sb, vb = random_operand(rng, n, k, spread=1.0, std=k ** -0.5)
    buf = sentinel(rows + 130, n).view(dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = moe.mx4_matmul(a, sa, b, sb, out=buf[:rows], status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert bool((buf[rows:].view(torch.int16) == SENTINEL).all())
    ref = va @ vb.t()
    check(out, ref, half_step(dt) * ref.abs() + tiny(dt) + 2 * acc(k) * (va.abs() @ vb.abs().t()), "matmul")
    again = moe.mx4_matmul(a, sa, b, sb, dtype=dt)
    assert torch.equal(again.view(torch.int16), out.contiguous().view(torch.int16))


@pytest.mark.parametrize("dt", OUT, ids=["fp16", "bf16"])
@pytest.mark.parametrize("rows,k,n", [(1, 3840, 128), (1, 4096, 128), (16, 4224, 640), (17, 4480, 256), (33, 6272, 384),
                                      (64, 4096, 4736), (65, 7168, 256), (100, 4096, 1152), (128, 4224, 384),
                                      (3, 4096, 4608), (2, 4096, 9856), (128, 4096, 2432)])
def test_matmul_few_rows_long_k(rows, k, n, dt):
    """Few rows against few weight slices: several blocks share a tile's K axis, unevenly too."""
    test_matmul(rows, k, n, dt)


def test_matmul_single_products():
    """One value a row: every pair of codes, at different places along K and scales, is exact."""
    k = 512
    codes = np.arange(16, dtype=np.uint8)
    for at in (0, 31, 63, 64, 127, 128, 200, 255, 256, 511):
        ca, cb = np.zeros((128, k), np.uint8), np.zeros((128, k), np.uint8)
        ca[:, at], cb[:, at] = np.resize(codes, 128), np.repeat(codes, 8)
        rng = np.random.default_rng(at)
        s_a = rng.integers(120, 130, (128, k // 32)).astype(np.uint8)
        s_b = rng.integers(120, 130, (128, k // 32)).astype(np.uint8)
        out = moe.mx4_matmul(torch.from_numpy(mx4_ref.pack(ca)).cuda(), torch.from_numpy(mx4_ref.tiles(s_a)).cuda(),
                             torch.from_numpy(mx4_ref.pack(cb)).cuda(), torch.from_numpy(mx4_ref.tiles(s_b)).cuda(),
                             dtype=torch.bfloat16)
        want = mx4_ref.values(ca, s_a) @ mx4_ref.values(cb, s_b).T
        assert np.array_equal(out.float().cpu().numpy().astype(np.float64), want), at


def test_nan_stays_in_its_row():
    rng = np.random.default_rng(1)
    a, sa, va = random_operand(rng, 140, 256)
    b, sb, vb = random_operand(rng, 256, 256)
    want = moe.mx4_matmul(a, sa, b, sb)
    s2 = sa.clone()
    s2[0, 1, 7, 2, 3] = 255                      # row 71, block 7
    got = moe.mx4_matmul(a, s2, b, sb)
    torch.cuda.synchronize()
    assert bool(got[71].isnan().all())
    keep = [r for r in range(140) if r != 71]
    assert torch.equal(got[keep], want[keep])


GROUPED = [  # tokens, top_k, experts, k, n, expert popularity exponent
    (1, 1, 1, 128, 128, 0.0), (1, 2, 4, 256, 256, 0.0), (5, 2, 8, 384, 384, 0.0), (40, 2, 4, 256, 640, 1.0),
    (130, 1, 2, 512, 128, 0.0), (300, 2, 3, 256, 384, 0.0), (600, 4, 8, 640, 256, 1.2), (33, 8, 128, 256, 256, 1.2),
    (1000, 1, 1, 1408, 512, 0.0), (700, 2, 64, 128, 896, 1.0),
    # one expert with few rows: the two halves of a block, and a short last one
    (64, 1, 1, 256, 128, 0.0), (65, 1, 1, 256, 256, 0.0), (127, 1, 1, 384, 128, 0.0), (128, 1, 1, 128, 128, 0.0),
    # many experts, some with several blocks, several groups of units
    (2600, 2, 3, 256, 640, 1.2), (400, 8, 256, 128, 128, 1.2)]


def grouped(T, top_k, E, seed, zipf):
    rng = np.random.default_rng(seed)
    keys = -zipf * np.log(np.arange(1, E + 1)) + rng.gumbel(size=(T, E))
    ids = torch.from_numpy(np.ascontiguousarray(np.argsort(-keys, axis=1)[:, :top_k].astype(np.int32))).cuda()
    w = torch.from_numpy(rng.random((T, top_k)).astype(np.float32)).cuda()
    t = moe.build_dispatch(ids, E)
    rows = t["group_idx_for_bx"].numel() * 128
    pk = moe.pack_routed(ids, w, None, t, rows)
    return rng, t, rows, pk["routed_expert_weights"], pk["pair_padded_rows"]


def row_experts(t, pair_rows):
    """The valid padded rows, each one's expert and compact index."""
    rows = pair_rows.reshape(-1).long().sort().values
    e = t["group_idx_for_bx"].long()[rows // 128]
    return rows, e, t["group_offsets"].long()[e] + rows - t["group_padded_offsets"].long()[e]


@pytest.mark.parametrize("dt", OUT, ids=["fp16", "bf16"])
@pytest.mark.parametrize("T,top_k,E,k,n,zipf", GROUPED)
def test_gate_up(T, top_k, E, k, n, zipf, dt):
    rng, t, rows, _, pr = grouped(T, top_k, E, T + k, zipf)
    a, sa, va = random_operand(rng, rows, k)
    g, sg, vg = random_operand(rng, E * n, k, std=k ** -0.5)
    u, su, vu = random_operand(rng, E * n, k, std=k ** -0.5)
    valid, e, _ = row_experts(t, pr)
    pad = torch.ones(rows, dtype=torch.bool, device="cuda")
    pad[valid] = False
    a[pad] = 0xFF                                 # padding rows hold anything, NaN scales among it
    r = torch.nonzero(pad).view(-1)
    sa[r // 128, :, r % 32, r // 32 % 4] = 255
    buf = sentinel(rows, n).view(dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.mx4_gate_up(a, sa, g.view(E, n, -1), sg, u.view(E, n, -1), su, t["group_sizes"], t["group_padded_offsets"],
                    t["group_idx_for_bx"], buf, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert bool((buf[pad].view(torch.int16) == SENTINEL).all())
    for ex in e.unique().tolist():
        x, wg, wu = va[valid[e == ex]], vg[ex * n:(ex + 1) * n], vu[ex * n:(ex + 1) * n]
        G, U = x @ wg.t(), x @ wu.t()
        dG, dU = acc(k) * (x.abs() @ wg.abs().t()), acc(k) * (x.abs() @ wu.abs().t())
        act = G * torch.sigmoid(G)
        ref = act * U
        off = 1.1 * U.abs() * dG + act.abs() * dU + 1.1 * dG * dU + 32 * 2.0 ** -23 * ref.abs()
        check(buf[valid[e == ex]], ref, half_step(dt) * ref.abs() + tiny(dt) + 2 * off, f"expert {ex}")


@pytest.mark.parametrize("dt", OUT, ids=["fp16", "bf16"])
@pytest.mark.parametrize("T,top_k,E,k,n,zipf", GROUPED)
def test_down(T, top_k, E, k, n, zipf, dt):
    rng, t, rows, w, pr = grouped(T, top_k, E, T + n, zipf)
    a, sa, va = random_operand(rng, rows, k)
    b, sb, vb = random_operand(rng, E * n, k, std=k ** -0.5)
    valid, e, compact = row_experts(t, pr)
    buf = sentinel(rows, n).view(dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.mx4_down(a, sa, b.view(E, n, -1), sb, w, t["group_sizes"], t["group_offsets"], t["group_padded_offsets"],
                 t["group_idx_for_bx"], buf, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    pad = torch.ones(rows, dtype=torch.bool, device="cuda")
    pad[valid] = False
    assert bool((buf[pad].view(torch.int16) == SENTINEL).all())
    for ex in e.unique().tolist():
        at = e == ex
        x, wd, rw = va[valid[at]], vb[ex * n:(ex + 1) * n], w[compact[at]].double()[:, None]
        ref = (x @ wd.t()) * rw
        tol = half_step(dt) * ref.abs() + tiny(dt) + 2 * acc(k) * (x.abs() @ wd.abs().t()) * rw + 2.0 ** -23 * ref.abs()
        check(buf[valid[at]], ref, tol, f"expert {ex}")


def test_bad_tables_are_reported():
    rng, t, rows, w, pr = grouped(300, 2, 4, 3, 0.0)
    a, sa, _ = random_operand(rng, rows, 256)
    b, sb, _ = random_operand(rng, 4 * 256, 256)
    want = sentinel(rows, 256)
    args = (a, sa, b.view(4, 256, -1), sb, w)
    tabs = [t[k] for k in ("group_sizes", "group_offsets", "group_padded_offsets", "group_idx_for_bx")]
    moe.mx4_down(*args, *tabs, want)
    for which, entry, value in ((3, 0, 4), (3, 0, -1), (1, 0, 1 << 20), (1, 0, -5)):
        bad = [v.clone() for v in tabs]
        bad[which][entry] = value
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = sentinel(rows, 256)
        moe.mx4_down(*args, *bad, got, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == moe.MOE_DEV_BAD_TABLE
        assert bool((got[:128].view(torch.int16) == SENTINEL).all())         # the block is left out
        first = 128 if which == 3 else int(t["group_padded_offsets"][1])     # offsets: every block of expert 0
        assert torch.equal(got[first:].view(torch.int16), want[first:].view(torch.int16))


def test_stream_and_graph():
    rng, t, rows, w, pr = grouped(200, 2, 4, 5, 0.0)
    x = torch.from_numpy(rng.standard_normal((rows, 256))).cuda().half()
    b, sb, _ = random_operand(rng, 4 * 128, 256)
    codes, scales = moe.mx4_quantize(x)
    out = sentinel(rows, 128)

    def step():
        moe.mx4_quantize(x, codes=codes, scales=scales)
        moe.mx4_down(codes, scales, b.view(4, 128, -1), sb, w, t["group_sizes"], t["group_offsets"],
                     t["group_padded_offsets"], t["group_idx_for_bx"], out)

    step()
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    out.zero_()
    codes.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    valid = pr.reshape(-1).long()
    assert torch.equal(out[valid], want[valid])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[valid], want[valid])


def test_refusals():
    x = torch.randn((4, 256), device="cuda").half()
    c, s = moe.mx4_quantize(x)
    with pytest.raises(ValueError, match="multiple of 128"):
        moe.mx4_quantize(x[:, :64].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        moe.mx4_quantize(x.t())
    with pytest.raises(ValueError, match="without row lists"):
        moe.mx4_quantize(x[None], src_rows=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="n_dest"):
        moe.mx4_quantize(x, dest_rows=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="dest_rows"):
        moe.mx4_quantize(x, dest_rows=torch.zeros(3, dtype=torch.int32, device="cuda"), n_dest=4)
    with pytest.raises(ValueError, match="codes"):
        moe.mx4_quantize(x, codes=c[:2])
    with pytest.raises(ValueError, match="must hold the tiles"):
        moe.mx4_dequantize(c, s[:, :1].contiguous(), torch.float16)
    with pytest.raises(TypeError, match="uint8"):
        moe.mx4_dequantize(c.int(), s, torch.float16)
    with pytest.raises(ValueError, match="same columns"):
        moe.mx4_matmul(c, s, *moe.mx4_quantize(torch.zeros((128, 128), device="cuda")))
    with pytest.raises(moe.MoeError, match="MOE_ERR_SHAPE"):
        moe.mx4_matmul(c, s, c, s)               # 4 columns of result
    w, ws = moe.mx4_quantize(torch.zeros((2, 128, 256), device="cuda"))
    t = moe.build_dispatch(torch.zeros((4, 1), dtype=torch.int32, device="cuda"), 2)
    tab = (t["group_sizes"], t["group_padded_offsets"], t["group_idx_for_bx"])
    with pytest.raises(moe.MoeError, match="MOE_ERR_SHAPE"):                 # 4 rows for 3 blocks
        moe.mx4_gate_up(c, s, w, ws, w, ws, *tab, torch.empty((4, 128), device="cuda").half())
    with pytest.raises(ValueError, match="up_logits"):
        moe.mx4_gate_up(c, s, w, ws, w, ws, *tab, torch.empty((4, 64), device="cuda").half())
    with pytest.raises(ValueError, match="n_experts"):
        moe.mx4_gate_up(c, s, w, ws, w, ws, tab[0][:1], *tab[1:], torch.empty((4, 128), device="cuda").half())


def test_no_rows():
    c, s = moe.mx4_quantize(torch.empty((0, 256), device="cuda"))
    assert c.shape == (0, 128) and s.shape == (0, 2, 32, 4, 4)
    assert moe.mx4_dequantize(c, s, torch.bfloat16).shape == (0, 256)
    b, sb = moe.mx4_quantize(torch.randn((128, 256), device="cuda"))
    assert moe.mx4_matmul(c, s, b, sb).shape == (0, 128)
    # tables without a pair
    t = moe.build_dispatch(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 3)
    rows = t["group_idx_for_bx"].numel() * 128
    a, sa = moe.mx4_quantize(torch.zeros((rows, 256), device="cuda"))
    out = sentinel(rows, 128)
    w, sw = moe.mx4_quantize(torch.zeros((3, 128, 256), device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.mx4_gate_up(a, sa, w, sw, w, sw, t["group_sizes"], t["group_padded_offsets"], t["group_idx_for_bx"], out, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and bool((out.view(torch.int16) == SENTINEL).all())


def test_offsets_past_32_bits():
    """Values past element 2^31: the last rows' results are those of a call on them alone."""
    rows, cols = (1 << 20) + 131, 2176
    assert rows * cols > 2 ** 31
    x = torch.zeros((rows, cols), dtype=torch.float16, device="cuda")
    last = rows - rows % 128 - 128                # a whole scale tile from here
    x[last:] = torch.randn((rows - last, cols), device="cuda").half()
    c, s = moe.mx4_quantize(x)
    want_c, want_s = moe.mx4_quantize(x[last:].contiguous())
    assert torch.equal(c[last:], want_c) and torch.equal(s[last // 128:], want_s)
    back = moe.mx4_dequantize(c, s, torch.float16)
    assert torch.equal(back[last:], moe.mx4_dequantize(want_c, want_s, torch.float16))
    assert not bool(back[:last].any())
    del x, c, s, back

    rows, k, n = 128 * 16384, 128, 1152            # the most blocks
    assert rows * n > 2 ** 31
    codes = torch.zeros((rows, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((rows // 128, 1, 32, 4, 4), 127, dtype=torch.uint8, device="cuda")
    codes[-300:] = torch.randint(0, 256, (300, k // 2), dtype=torch.uint8, device="cuda")
    b, sb = moe.mx4_quantize(torch.randn((n, k), device="cuda"))
    out = moe.mx4_matmul(codes, scales, b, sb)
    want = moe.mx4_matmul(codes[-384:].contiguous(), scales[-3:].contiguous(), b, sb)
    torch.cuda.synchronize()
    assert torch.equal(out[-384:], want)
    assert not bool(out[:-384].any())
