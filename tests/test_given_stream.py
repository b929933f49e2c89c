"""Memory that a call allocates and uses on a given stream stays its own until that stream is done.

Without a device: every tensor that the binding allocates for a call is recorded on the given stream,
whatever form that has.  On one: results of calls chained on a busy stream, whose intermediate tensors
are dropped and asked for again on the current stream meanwhile."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import routed_grouped_gemm_dispatch_gb300 as moe


class NoLibrary:
    """Takes every call and says that it went well."""

    def __getattr__(self, name):
        return lambda *a: 1 if name.endswith(("_bytes", "_blocks")) else 0


def calls():
    """Every call that takes a stream, with what it needs and nothing that it can allocate itself."""
    def t(*shape, dt=torch.float16):
        return torch.empty(shape, dtype=dt, device="cuda")

    i32, u8, f32 = torch.int32, torch.uint8, torch.float32
    x, w, d = t(4, 128), t(256, 128), t(128, 256)
    h = t(4, 256)
    c, s = t(128, 64, dt=u8), t(1, 1, 32, 4, 4, dt=u8)
    tables = {"group_sizes": t(2, dt=i32), "group_offsets": t(3, dt=i32), "group_padded_offsets": t(3, dt=i32),
              "group_idx_for_bx": t(3, dt=i32)}
    return {
        "build_dispatch": ((t(4, 2, dt=i32), 2), 4),
        "pack_routed": ((t(4, 2, dt=i32), t(4, 2, dt=f32), x, tables), 4),
        "combine_routed": ((t(384, 128), t(4, 2, dt=i32)), 1),
        "router_topk": ((x, t(2, 128), 1), 2),
        "gated_ffn": ((x, w, w, d), 2),
        "gated_ffn_backward": ((x, x, w, w, d, h, h, h), 5),
        "mx4_quantize": ((x,), 2),
        "mx4_dequantize": ((c, s, torch.float16), 1),
        "mx4_matmul": ((c, s, c, s), 1),
    }


@pytest.mark.parametrize("kind", ["object", "handle", "default", None])
@pytest.mark.parametrize("name", ["build_dispatch", "pack_routed", "combine_routed", "router_topk", "gated_ffn",
                                  "gated_ffn_backward", "mx4_quantize", "mx4_dequantize", "mx4_matmul"])
def test_allocations_are_recorded(name, kind, monkeypatch):
    class Stream:
        cuda_stream = 0x77

    made, recorded = [], []
    monkeypatch.setattr(moe, "lib", lambda lib=NoLibrary(): lib)
    monkeypatch.setattr(moe, "_stream", lambda s: 0 if s is None else getattr(s, "cuda_stream", s))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda p, device=None: ("handle", p))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("handle", 0))
    stream, want = {"object": (s := Stream(), s), "handle": (0x99, ("handle", 0x99)), "default": (0, ("handle", 0)),
                    None: (None, None)}[kind]
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")          # tensors without data have no address
        args, n = calls()[name]
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((id(t), s)))
        inside = []                              # full may be made of an empty
        for f in ("empty", "empty_like", "full"):
            def spy(*a, _f=getattr(torch, f), **k):
                inside.append(1)
                r = _f(*a, **k)
                inside.pop()
                if not inside:
                    made.append(r)
                return r
            monkeypatch.setattr(torch, f, spy)
        getattr(moe, name)(*args, stream=stream)
    assert len(made) == n
    assert recorded == ([] if kind is None else [(id(t), want) for t in made])


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["object", "handle"])
def test_chain_on_a_busy_stream(form):
    """Quantise and multiply on a stream that has other work first; codes and scales are dropped at once."""
    x, b = torch.randn((300, 512), device="cuda").half(), torch.randn((256, 512), device="cuda").half()
    bq, bs = moe.mx4_quantize(b)
    want = moe.mx4_matmul(*moe.mx4_quantize(x), bq, bs)
    back = moe.mx4_dequantize(*moe.mx4_quantize(x), torch.float16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side if form == "object" else side.cuda_stream
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)        # about 10 ms
        got = moe.mx4_matmul(*moe.mx4_quantize(x, stream=stream), bq, bs, stream=stream)
        again = moe.mx4_dequantize(*moe.mx4_quantize(x, stream=stream), torch.float16, stream=stream)
        for _ in range(8):                       # what would take the dropped codes and scales
            torch.full((300, 256), 0xFF, dtype=torch.uint8, device="cuda")
            torch.full((3, 4, 32, 4, 4), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        assert torch.equal(again.view(torch.int16), back.view(torch.int16))
