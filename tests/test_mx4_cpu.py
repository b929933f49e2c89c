"""The 4-bit definition itself against hand-worked values, and the host-side refusals."""
import numpy as np
import pytest
import torch

import mx4_ref
import routed_grouped_gemm_dispatch_gb300 as moe


def test_definition_by_hand():
    x = np.zeros((1, 64))
    # amax 7.9 -> floor(log2) = 2, e = 0: every tie goes to the even code, 5 < x saturates at 6
    x[0, :12] = [7.9, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, -0.25, -6.0]
    # amax 0.24 -> floor(log2) = -3, e = -5
    x[0, 32:35] = [0.24, -0.125, 0.0]
    codes, scales = mx4_ref.quantize(x)
    assert codes[0, :12].tolist() == [7, 0, 1, 2, 2, 4, 4, 6, 6, 7, 8, 15]
    assert scales[0].tolist() == [127, 122]
    assert codes[0, 32:35].tolist() == [7, 14, 0]            # 7.68 -> 6, -4, 0
    v = mx4_ref.values(codes, scales)
    assert v[0, 0] == 6 and v[0, 32] == 6 / 32 and v[0, 33] == -0.125
    bad = np.zeros((1, 32))
    bad[0, 3] = np.inf
    bad[0, 4] = -1
    codes, scales = mx4_ref.quantize(bad)
    assert scales[0, 0] == 255 and not codes.any()


def test_tiles_round_trip():
    s = np.arange(130 * 8, dtype=np.int64).reshape(130, 8).astype(np.uint8)
    t = mx4_ref.tiles(s)
    assert t.shape == (2, 2, 32, 4, 4)
    assert (mx4_ref.untile(t, 130) == s).all()
    # row 70, block 5 by the formula
    assert t[0, 1, 70 % 32, 2, 1] == s[70, 5]


@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


def test_quantize_refusals(L):
    base = dict(dt=0, x=0x1000, ns=5, cols=256, src=None, n=5, dst=None, copies=1, nd=5, codes=0x2000, scales=0x3000)

    def call(**kw):
        a = {**base, **kw}
        return L.moe_mx4_quantize(a["dt"], a["x"], a["ns"], a["cols"], a["src"], a["n"], a["dst"], a["copies"], a["nd"],
                                  a["codes"], a["scales"], None, None)

    assert call(dt=3) == -2 and call(dt=-1) == -2
    assert call(cols=192) == -2 and call(cols=0) == -2 and call(cols=(1 << 17) + 128) == -7
    assert call(ns=-1, n=-1, nd=-1) == -2
    assert call(n=4) == -2                       # without src_rows every row is converted
    assert call(src=0x4000, n=4) == -2           # without dest_rows the result has the converted rows
    assert call(copies=0) == -2 and call(copies=2) == -2
    assert call(ns=(1 << 24) + 1, n=(1 << 24) + 1, nd=(1 << 24) + 1) == -7
    assert call(x=None) == -1 and call(codes=None) == -1 and call(scales=None) == -1
    assert call(x=0x1008) == -3 and call(codes=0x2008) == -3 and call(scales=0x3001) == -3
    assert call(ns=0, n=0, nd=0, x=None) == 0
    assert L.moe_mx4_scale_bytes(129, 256) == 2 * 2 * 512
    assert L.moe_mx4_scale_bytes(0, 256) == 0
    assert L.moe_mx4_scale_bytes(1, 100) == -1
    assert L.moe_mx4_dequantize(0x1000, 0x2000, 5, 256, 4, 0x3000, None) == -2
    assert L.moe_mx4_dequantize(0x1000, 0x2000, 5, 250, 0, 0x3000, None) == -2
    assert L.moe_mx4_dequantize(0x1000, None, 5, 256, 0, 0x3000, None) == -1
    assert L.moe_mx4_dequantize(0x1000, 0x2000, 5, 256, 0, 0x3008, None) == -3


def test_product_refusals(L):
    def matmul(a=0x1000, s=0x2000, rows=5, k=256, b=0x3000, bs=0x4000, n=128, dt=0, out=0x5000):
        return L.moe_mx4_matmul(a, s, rows, k, b, bs, n, dt, out, None, None)

    assert matmul(dt=2) == -2 and matmul(k=64) == -2 and matmul(n=100) == -2 and matmul(rows=-1) == -2
    assert matmul(rows=128 * 16384 + 1) == -7 and matmul(n=(1 << 17) + 128) == -7
    for k in ("a", "s", "b", "bs", "out"):
        assert matmul(**{k: None}) == -1 and matmul(**{k: 0x1008}) == -3, k
    assert matmul(rows=0, a=None, out=None) == 0

    def gate_up(x=0x1000, xs=0x2000, rows=640, H=256, g=0x3000, gs=0x4000, u=0x5000, us=0x6000, E=4, I=128, sz=0x7000,
                pad=0x8000, gi=0x9000, m=5, dt=1, out=0xA000):
        return L.moe_mx4_gate_up(x, xs, rows, H, g, gs, u, us, E, I, sz, pad, gi, m, dt, out, None, None)

    assert gate_up(dt=2) == -2 and gate_up(H=100) == -2 and gate_up(I=0) == -2
    assert gate_up(rows=639) == -2               # fewer rows than blocks
    assert gate_up(E=0) == -7 and gate_up(E=1025) == -7 and gate_up(m=20000, rows=20000 * 128) == -7
    assert gate_up(E=1024, I=128 * 1024) == -7   # more weight rows than a 4-bit array holds
    for k in ("x", "xs", "g", "gs", "u", "us", "out"):
        assert gate_up(**{k: None}) == -1 and gate_up(**{k: 0x1004}) == -3, k
    for k in ("sz", "pad", "gi"):
        assert gate_up(**{k: None}) == -1, k

    def down(h=0x1000, hs=0x2000, rows=640, I=256, d=0x3000, ds=0x4000, E=4, H=128, w=0x5000, nv=100, sz=0x7000,
             off=0x6000, pad=0x8000, gi=0x9000, m=5, dt=1, out=0xA000):
        return L.moe_mx4_down(h, hs, rows, I, d, ds, E, H, w, nv, sz, off, pad, gi, m, dt, out, None, None)

    assert down(nv=-1) == -2 and down(H=64) == -2 and down(m=-1) == -2
    for k in ("h", "hs", "d", "ds", "out", "w", "sz", "off", "pad", "gi"):
        assert down(**{k: None}) == -1, k


def test_binding_refusals(L):
    x = torch.zeros((4, 128), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.mx4_quantize(x)
    with pytest.raises(TypeError, match="float32"):
        moe.mx4_quantize(x.double())
    with pytest.raises(TypeError):
        moe.mx4_quantize(None)
    with pytest.raises(ValueError, match="CUDA"):
        moe.mx4_dequantize(torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((1, 1, 32, 4, 4), dtype=torch.uint8),
                           torch.float16)
