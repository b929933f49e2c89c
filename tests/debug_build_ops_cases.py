"""Feed-forward and 4-bit cases that tests/test_debug_build_ops_gpu.py runs twice: in the test
process with the release library, and in a child process started with MOE_GB300_DEBUG=1, which
loads the MOE_DEBUG build.  Every output and every status word goes into one .npz per run.

    python debug_build_ops_cases.py OUT.npz
"""
import sys

import numpy as np
import torch

import routed_grouped_gemm_dispatch_gb300 as moe
from gpu_side import bits, sentinel

# one token to several tiles; tiles shared by two, three and four pairs; d_down in either launch
FFN = [(1, 8, 8), (37, 264, 392), (128, 520, 136), (129, 384, 640), (200, 4104, 136), (260, 520, 2056), (301, 2048, 2816),
       (520, 1544, 1288), (1025, 904, 2056), (32, 1032, 776), (448, 384, 7176)]
# rows, k, n: one block and several, K shared among blocks, a last slice of half a tile
MATMUL = [(1, 256, 128), (65, 4096, 256), (17, 4480, 256), (128, 1408, 384), (129, 2048, 384), (1111, 512, 640)]
# tokens, top_k, experts, k, n
GROUPED = [(5, 2, 8, 384, 384), (300, 2, 3, 256, 384), (33, 8, 128, 256, 256), (1000, 1, 1, 1408, 512), (2600, 2, 3, 256, 640)]


def run_cases():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def draw(*shape, dt=torch.float16):
        return torch.randn(shape, generator=g, device="cuda").mul_(shape[-1] ** -0.5).to(dt)

    res = {}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for T, H, I in FFN:
        for dt in (torch.float16, torch.bfloat16):
            x, d_out, gate_w, up_w, down_w = draw(T, H, dt=dt) * 4, draw(T, H, dt=dt), draw(I, H, dt=dt), draw(I, H, dt=dt), draw(H, I, dt=dt)
            s = {k: torch.empty((T, I), dtype=dt, device="cuda") for k in ("gate", "up", "up_logits")}
            out = moe.gated_ffn(x, gate_w, up_w, down_w, status=status, **s)
            grads = moe.gated_ffn_backward(d_out, x, gate_w, up_w, down_w, s["gate"], s["up"], s["up_logits"], status=status)
            for k, t in {**s, "out": out, **{f"grad{i}": t for i, t in enumerate(grads)}}.items():
                res[f"ffn {T} {H} {I} {dt}/{k}"] = bits(t)
    res["ffn/status"] = status.cpu().numpy().copy()
    status.zero_()
    for rows, k, n in MATMUL:
        a, b = moe.mx4_quantize(draw(rows, k), status=status), moe.mx4_quantize(draw(n, k), status=status)
        res[f"matmul {rows} {k} {n}/codes"], res[f"matmul {rows} {k} {n}/scales"] = (t.cpu().numpy() for t in a)
        res[f"matmul {rows} {k} {n}/out"] = bits(moe.mx4_matmul(*a, *b, status=status))
        res[f"matmul {rows} {k} {n}/back"] = bits(moe.mx4_dequantize(*a, torch.float16))
    for T, top_k, E, k, n in GROUPED:
        ids = torch.rand((T, E), generator=g, device="cuda").argsort(dim=1)[:, :top_k].to(torch.int32).contiguous()
        t = moe.build_dispatch(ids, E)
        rows = t["group_idx_for_bx"].numel() * 128
        p = moe.pack_routed(ids, torch.rand((T, top_k), generator=g, device="cuda"), None, t, rows)
        x = draw(T, k) * 4
        codes = torch.zeros((rows, k // 2), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((rows // 128, k // 128, 32, 4, 4), dtype=torch.uint8, device="cuda")
        moe.mx4_quantize(x, dest_rows=p["pair_padded_rows"], codes=codes, scales=scales, status=status)
        gate, up = moe.mx4_quantize(draw(E, n, k), status=status), moe.mx4_quantize(draw(E, n, k), status=status)
        tabs = [t[v] for v in ("group_sizes", "group_offsets", "group_padded_offsets", "group_idx_for_bx")]
        h, o = sentinel(rows, n), sentinel(rows, n)
        moe.mx4_gate_up(codes, scales, *gate, *up, tabs[0], tabs[2], tabs[3], h, status=status)
        moe.mx4_down(codes, scales, *up, p["routed_expert_weights"], *tabs, o, status=status)
        picked = moe.mx4_quantize(x, src_rows=torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda"), status=status)
        name = f"grouped {T} {top_k} {E} {k} {n}"
        res[f"{name}/codes"], res[f"{name}/scales"] = codes.cpu().numpy(), scales.cpu().numpy()
        res[f"{name}/h"], res[f"{name}/o"] = bits(h), bits(o)
        res[f"{name}/picked"], res[f"{name}/picked scales"] = (v.cpu().numpy() for v in picked)
    torch.cuda.synchronize()
    res["mx4/status"] = status.cpu().numpy().copy()
    return res


if __name__ == "__main__":
    np.savez(sys.argv[1], **run_cases())
