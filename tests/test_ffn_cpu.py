"""Refusals of the dense feed-forward block: every call here fails a check on the
host, before anything is enqueued."""
import pytest
import torch

import routed_grouped_gemm_dispatch_gb300 as moe


@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


FWD = dict(dtype=0, x=0x1000, T=5, H=64, g=0x2000, u=0x3000, d=0x4000, I=72, gate=0x5000, up=0x6000, ul=0x7000,
           out=0x8000)


def fwd(L, **kw):
    a = {**FWD, **kw}
    return L.moe_ffn_forward(a["dtype"], a["x"], a["T"], a["H"], a["g"], a["u"], a["d"], a["I"], a["gate"], a["up"],
                             a["ul"], a["out"], None, None)


BWD = dict(dtype=1, dy=0x1000, x=0x2000, T=5, H=64, g=0x3000, u=0x4000, d=0x5000, I=72, gate=0x6000, up=0x7000,
           ul=0x8000, ws=0x9000, n=1 << 20, dx=0xA000, dg=0xB000, du=0xC000, dd=0xD000)


def bwd(L, **kw):
    a = {**BWD, **kw}
    return L.moe_ffn_backward(a["dtype"], a["dy"], a["x"], a["T"], a["H"], a["g"], a["u"], a["d"], a["I"], a["gate"],
                              a["up"], a["ul"], a["ws"], a["n"], a["dx"], a["dg"], a["du"], a["dd"], None, None)


def test_forward_refusals(L):
    assert fwd(L, dtype=2) == -2
    assert fwd(L, dtype=-1) == -2
    assert fwd(L, T=-1) == -2
    assert fwd(L, H=0) == -2
    assert fwd(L, H=60) == -2                 # rows must be whole 16-byte pieces
    assert fwd(L, I=4) == -2
    assert fwd(L, T=(1 << 24) + 1) == -7
    assert fwd(L, H=(1 << 20) + 8) == -7
    assert fwd(L, I=(1 << 20) + 8) == -7
    for k in ("x", "g", "u", "d", "ul", "out", "gate", "up"):   # gate without up, up without gate
        assert fwd(L, **{k: None}) == -1, k
    for k in ("x", "g", "u", "d", "ul", "out", "gate", "up"):
        assert fwd(L, **{k: 0x1008}) == -3, k
    assert fwd(L, T=0, x=None, out=None) == 0                    # nothing to do


def test_backward_refusals(L):
    assert bwd(L, dtype=2) == -2
    assert bwd(L, T=-1) == -2
    assert bwd(L, H=12) == -2
    assert bwd(L, I=0) == -2
    assert bwd(L, T=(1 << 24) + 1) == -7
    for k in ("dy", "x", "g", "u", "d", "gate", "up", "ul", "dx", "dg", "du", "dd"):
        assert bwd(L, **{k: None}) == -1, k
        assert bwd(L, **{k: 0x1004}) == -3, k
    assert bwd(L, ws=None) == -8
    assert bwd(L, n=2 * 768 - 1) == -8        # two arrays of 5 * 72 * 2 bytes, each rounded up to 256
    assert bwd(L, ws=0x9008) == -3
    assert L.moe_ffn_backward_workspace_bytes(5, 72) == 2 * 768
    assert L.moe_ffn_backward_workspace_bytes(-1, 72) == -1
    assert L.moe_ffn_backward_workspace_bytes(1 << 24, 1 << 20) == 1 << 46


def test_binding_refusals(L):
    x = torch.zeros((3, 16), dtype=torch.float16)
    w = torch.zeros((8, 16), dtype=torch.float16)
    d = torch.zeros((16, 8), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.gated_ffn(x, w, w, d)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        moe.gated_ffn(x.float(), w, w, d)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        moe.gated_ffn(None, w, w, d)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        moe.gated_ffn_backward(x.double(), x.double(), w, w, d, x, x, x)
