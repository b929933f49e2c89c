"""Cases of the training operators that tests/test_debug_build_train_gpu.py runs twice: in the test process with the
release library, and in a child process started with MOE_GB300_DEBUG=1, which loads the MOE_DEBUG build.  Every
output and every status word goes into one .npz per run.

    python debug_build_train_cases.py OUT.npz
"""
import sys

import numpy as np
import torch

import routed_grouped_gemm_dispatch_gb300 as moe

# tokens, experts, top_k, hidden, sequences, masked: one block and many, whole tiles of d_W and parts, one to four rows of them
ROUTER = [(1, 4, 2, 8, 1, False), (33, 130, 8, 520, 3, True), (300, 1021, 16, 768, 4, True), (2049, 64, 6, 2048, 5, True),
          (5000, 256, 8, 1032, 1, False), (700, 33, 2, 4104, 1, False)]
# batch, rows, cols: one cluster, and tiles of either width
ORTHO = [(1, 1, 1), (3, 100, 700), (2, 128, 128), (1, 130, 6200), (1, 333, 1001), (2, 700, 300), (20, 520, 600), (1, 1500, 2100)]


def run_cases():
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    res = {}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for T, E, k, H, seqs, masked in ROUTER:
        z = torch.randn((T, E), generator=g, device="cuda")
        ids = torch.topk(z, k, dim=1).indices.to(torch.int32)
        kw = {"status": status}
        if seqs > 1:
            cuts = torch.randint(0, T + 1, (seqs - 1,), generator=g, device="cuda").sort().values
            kw["seq_offsets"] = torch.cat((torch.zeros_like(cuts[:1]), cuts, torch.full_like(cuts[:1], T))).to(torch.int32)
        if masked:
            kw["token_mask"] = torch.rand((T,), generator=g, device="cuda") >= 0.2
        losses, counts, tokens = moe.router_balance(z, ids, **kw)
        dw, dl = torch.randn((T, k), generator=g, device="cuda"), torch.tensor([2.0, 0.25], device="cuda")
        for dt in (torch.float16, torch.bfloat16):
            x, w = (torch.randn(s, generator=g, device="cuda").to(dt) for s in ((T, H), (E, H)))
            if masked:
                x[~kw["token_mask"]] = float("nan")
            got = moe.router_backward(x, w, z, ids, dw, dl, counts, tokens, **kw)
            for i, t in enumerate((losses, counts, tokens, *got)):
                res[f"router {T} {E} {H} {dt}/{i}"] = t.view(torch.int16 if t.element_size() == 2 else torch.int32).cpu().numpy()
    torch.cuda.synchronize()
    res["router/status"] = status.cpu().numpy().copy()
    status.zero_()
    for batch, rows, cols in ORTHO:
        for dt in (torch.float16, torch.bfloat16, torch.float32):
            u = torch.randn((batch, rows, cols), generator=g, device="cuda").to(dt)
            res[f"ortho {batch} {rows} {cols} {dt}"] = moe.orthogonalize(u, status=status).view(torch.int16).cpu().numpy()
    torch.cuda.synchronize()
    res["ortho/status"] = status.cpu().numpy().copy()
    return res


if __name__ == "__main__":
    np.savez(sys.argv[1], **run_cases())
