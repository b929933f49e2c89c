"""Python binding of the routed fused-MoE expert GEMM library (GB300, sm_103a).

Argument marshalling only: every step runs in the CUDA library
``_build/libmoe_gb300.so`` through its C ABI (``include/moe_gb300.h``).
PyTorch provides device memory and the current stream.  There is no CPU or
PyTorch fallback: if the library is missing or the device is not an sm_103
part, every call raises.

Calls (names follow "Fused MoE GEMM 提交说明", §提交文件 / §完整算子代码, and
"moe_dispatch_contract.py"):

  build_dispatch(topk_ids, n_experts)           -> dict of the four int32 tables
  fused_forward(stacked_expert_tokens, gate_w, up_w, down_w,
                routed_expert_weights, group_sizes, group_offsets,
                group_padded_offsets, group_idx_for_bx, up_logits, out)
  run_kernel(...)                               the page's signature (no up_logits;
                                                a cached workspace is used)
  pack_routed(topk_ids, topk_weights, x_tokens, tables)  -> grouped, padded inputs
  combine_routed(out, pair_rows)                -> token-major sum of the expert rows
  router_topk(x_tokens, router_w, top_k)        -> topk_ids, topk_weights

The dense gated feed-forward block (fp16 or bf16):

  gated_ffn(x, gate_w, up_w, down_w)            -> out (and, into given buffers, what the backward reads)
  gated_ffn_backward(d_out, x, gate_w, up_w, down_w, gate, up, up_logits)
                                                -> d_x, d_gate_w, d_up_w, d_down_w

Training of a routed layer:

  router_balance(logits, topk_ids)              -> losses, counts, seq_tokens
  router_backward(x_tokens, router_w, logits, topk_ids, ...)
                                                -> d_x, d_router_w
  orthogonalize(update)                         -> the update with singular values near 1

4-bit microscaled values (codes and scales) and products of them:

  mx4_quantize(x)                               -> codes, scales
  mx4_dequantize(codes, scales, dtype)          -> the values they stand for
  mx4_matmul(a, a_scales, b, b_scales)          -> a·bᵀ
  mx4_gate_up(...), mx4_down(...)               the routed experts' two halves, in the
                                                layout and with the tables of fused_forward

Work goes to the current stream, or to the ``stream`` that a call is given (an
object with cuda_stream, or the handle).  What a call allocates comes from the
current stream's memory, so a given stream has to wait for the current one
first; it is not handed out again before the given stream is done with it.
"""
from __future__ import annotations

import ctypes
import os
import threading

BLOCK_TOKEN = 128
MAX_EXPERTS = 1024          # MOE_MAX_EXPERTS
MAX_BLOCKS = 16384          # MOE_MAX_BLOCKS
ROUTER_MAX_EXPERTS = 256    # MOE_ROUTER_MAX_EXPERTS
ROUTER_MAX_TOPK = 16        # MOE_ROUTER_MAX_TOPK

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_GB300_DEBUG=1 in the environment selects the MOE_DEBUG build (kernels
# that also check their own indices and report MOE_DEV_DEBUG_CHECK).
LIB_PATH = os.path.join(_PKG, "_build", "libmoe_gb300_debug.so" if os.environ.get("MOE_GB300_DEBUG") == "1"
                        else "libmoe_gb300.so")

MOE_OK = 0
MOE_DEV_BAD_EXPERT_ID = 0x1
MOE_DEV_BAD_TABLE = 0x2
MOE_DEV_TIMEOUT = 0x4
MOE_DEV_DEBUG_CHECK = 0x8
MOE_RUN_PHASE1 = 0x1
MOE_RUN_PHASE2 = 0x2
MOE_NO_PDL = 0x4
MOE_TEST_DROP_SIGNAL = 0x100
MOE_DTYPE_F16 = 0
MOE_DTYPE_BF16 = 1
MOE_DTYPE_F32 = 2

_lock = threading.Lock()
_lib = None


class MoeError(RuntimeError):
    """A call of the C ABI returned a MOE_ERR_* status."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def build(force: bool = False, debug: bool = False) -> str:
    """Compile the CUDA library in-tree (nvcc, sm_103a); debug=True builds the
    MOE_DEBUG variant."""
    from . import _build
    return _build.build(force=force, debug=debug)


def lib():
    """The loaded C library; raises if it has not been built."""
    global _lib
    L = _lib
    if L is not None:
        return L
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built ({LIB_PATH}); call build() first")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.moe_abi_version.argtypes = []
        L.moe_abi_version.restype = i32
        L.moe_status_string.argtypes = [i32]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_num_blocks.argtypes = [i64, i32, i32]
        L.moe_num_blocks.restype = i64
        L.moe_build_dispatch.argtypes = [P, i64, i32, i32, i32, P, P, P, P, i64, P, P]
        L.moe_build_dispatch.restype = i32
        L.moe_fused_forward.argtypes = [P, i64, i32, P, P, P, i32, i32, P, i64,
                                        P, P, P, P, i64, P, P, P, P]
        L.moe_fused_forward.restype = i32
        L.moe_fused_forward_ex.argtypes = L.moe_fused_forward.argtypes + [ctypes.c_uint32]
        L.moe_fused_forward_ex.restype = i32
        L.moe_fused_forward_static_workspace.argtypes = [P, i64, i32, P, P, P, i32, i32, P, i64,
                                                         P, P, P, P, i64, P, P, P]
        L.moe_fused_forward_static_workspace.restype = i32
        L.moe_pack_workspace_bytes.argtypes = [i64, i32]
        L.moe_pack_workspace_bytes.restype = i64
        L.moe_pack_routed.argtypes = [P, P, i64, i32, i32, P, i32, P, P, i64, P, P, P, P,
                                      ctypes.c_size_t, P, P]
        L.moe_pack_routed.restype = i32
        L.moe_combine_routed.argtypes = [P, i64, i32, P, i64, i32, P, P]
        L.moe_combine_routed.restype = i32
        L.moe_router_topk.argtypes = [P, i64, i32, P, i32, i32, P, P, P, P]
        L.moe_router_topk.restype = i32
        L.moe_router_topk_logits.argtypes = [P, i64, i32, P, i32, i32, P, P, P, P, P]
        L.moe_router_topk_logits.restype = i32
        L.moe_router_balance_workspace_bytes.argtypes = [i64, i32, i32]
        L.moe_router_balance_workspace_bytes.restype = i64
        L.moe_router_balance.argtypes = [P, P, i64, i32, i32, P, P, i32, P, P, P, P, ctypes.c_size_t, P, P]
        L.moe_router_balance.restype = i32
        L.moe_router_backward_workspace_bytes.argtypes = [i64, i32, i32]
        L.moe_router_backward_workspace_bytes.restype = i64
        L.moe_router_backward.argtypes = [i32, P, i64, i32, P, i32, P, P, i32, P, P, P, P, P, P, i32, P,
                                          ctypes.c_size_t, P, P, P, P, P]
        L.moe_router_backward.restype = i32
        L.moe_orthogonalize_workspace_bytes.argtypes = [i64, i32, i32]
        L.moe_orthogonalize_workspace_bytes.restype = i64
        L.moe_orthogonalize.argtypes = [i32, P, i64, i32, i32, i32, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                        ctypes.c_float, P, ctypes.c_size_t, P, P, P]
        L.moe_orthogonalize.restype = i32
        L.moe_single_launch_workspace_bytes.argtypes = [i64]
        L.moe_single_launch_workspace_bytes.restype = i64
        L.moe_fused_forward_single_launch.argtypes = [P, i64, i32, P, P, P, i32, i32, P, i64,
                                                      P, P, P, P, i64, P, P, P, ctypes.c_size_t, P, P]
        L.moe_fused_forward_single_launch.restype = i32
        L.moe_ffn_forward.argtypes = [i32, P, i64, i32, P, P, P, i32, P, P, P, P, P, P]
        L.moe_ffn_forward.restype = i32
        L.moe_ffn_backward_workspace_bytes.argtypes = [i64, i32]
        L.moe_ffn_backward_workspace_bytes.restype = i64
        L.moe_ffn_backward.argtypes = [i32, P, P, i64, i32, P, P, P, i32, P, P, P, P, ctypes.c_size_t,
                                       P, P, P, P, P, P]
        L.moe_ffn_backward.restype = i32
        L.moe_mx4_scale_bytes.argtypes = [i64, i32]
        L.moe_mx4_scale_bytes.restype = i64
        L.moe_mx4_quantize.argtypes = [i32, P, i64, i32, P, i64, P, i32, i64, P, P, P, P]
        L.moe_mx4_quantize.restype = i32
        L.moe_mx4_dequantize.argtypes = [P, P, i64, i32, i32, P, P]
        L.moe_mx4_dequantize.restype = i32
        L.moe_mx4_matmul.argtypes = [P, P, i64, i32, P, P, i32, i32, P, P, P]
        L.moe_mx4_matmul.restype = i32
        L.moe_mx4_gate_up.argtypes = [P, P, i64, i32, P, P, P, P, i32, i32, P, P, P, i64, i32, P, P, P]
        L.moe_mx4_gate_up.restype = i32
        L.moe_mx4_down.argtypes = [P, P, i64, i32, P, P, i32, i32, P, i64, P, P, P, P, i64, i32, P, P, P]
        L.moe_mx4_down.restype = i32
        _lib = L
        return L


def single_launch_workspace_bytes(num_blocks_m: int) -> int:
    return int(lib().moe_single_launch_workspace_bytes(int(num_blocks_m)))


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def num_blocks(pairs: int, n_experts: int, block_token: int = BLOCK_TOKEN) -> int:
    return int(lib().moe_num_blocks(int(pairs), int(n_experts), int(block_token)))


def _stream(stream):
    import torch
    if stream is None:
        # the current stream's handle without building a Stream object (the
        # call Triton uses too); the public query where it does not exist
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _used_on(stream, *tensors):
    """Keep tensors that a call allocated from being handed out again before
    ``stream``'s work on them is done."""
    if stream is None:
        return
    import torch
    for t in tensors:
        s = stream
        if not hasattr(s, "cuda_stream"):        # a handle; 0 is the default stream's
            s = torch.cuda.ExternalStream(s, t.device) if s else torch.cuda.default_stream(t.device)
        t.record_stream(s)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dev(t, name, dtype, ndim=None):
    import torch
    # the common case in one expression; the checks below name what is wrong
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and (ndim is None or t.dim() == ndim)
            and t.is_contiguous()):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    return t


def _status(t):
    """Address of a status word that was given, an int32 on the device."""
    if t is None:
        return None
    import torch
    if not _dev(t, "status", torch.int32).numel():
        raise ValueError("status must hold an element")
    return t.data_ptr()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def build_dispatch(topk_ids, n_experts: int, block_token: int = BLOCK_TOKEN,
                   status=None, stream=None, out=None) -> dict:
    """The four dispatch tables for ``topk_ids`` [T, k] int32 (device).

    ``out`` may supply preallocated tables (same keys as the result)."""
    import torch
    ids = _dev(topk_ids, "topk_ids", torch.int32, 2)
    T, k = ids.shape
    E = int(n_experts)
    m = num_blocks(T * k, E, block_token)
    if out is None:
        dev = ids.device
        out = {
            "group_sizes": torch.empty(E, dtype=torch.int32, device=dev),
            "group_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
            "group_padded_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
            "group_idx_for_bx": torch.empty(max(m, 0), dtype=torch.int32, device=dev),
        }
        _used_on(stream, *out.values())
    st = lib().moe_build_dispatch(
        _ptr(ids), T, k, E, int(block_token), _ptr(out["group_sizes"]), _ptr(out["group_offsets"]),
        _ptr(out["group_padded_offsets"]), _ptr(out["group_idx_for_bx"]), m,
        _ptr(status), _stream(stream))
    _check(st, "moe_build_dispatch")
    return out


def fused_forward(stacked_expert_tokens, gate_w, up_w, down_w, routed_expert_weights,
                  group_sizes, group_offsets, group_padded_offsets, group_idx_for_bx,
                  up_logits, out, status=None, stream=None,
                  flags: int = MOE_RUN_PHASE1 | MOE_RUN_PHASE2, single_launch_workspace=None):
    """Phase 1 + phase 2 on the current stream; writes ``up_logits`` and ``out``
    in place on valid rows only.  ``flags`` selects phases (MOE_RUN_PHASE1 /
    MOE_RUN_PHASE2, optionally MOE_NO_PDL).  With ``single_launch_workspace``
    (a device tensor of at least single_launch_workspace_bytes() bytes) both
    phases run in one persistent launch."""
    import torch
    x = _dev(stacked_expert_tokens, "stacked_expert_tokens", torch.float16, 2)
    g = _dev(gate_w, "gate_w", torch.float16, 3)
    u = _dev(up_w, "up_w", torch.float16, 3)
    d = _dev(down_w, "down_w", torch.float16, 3)
    rw = _dev(routed_expert_weights, "routed_expert_weights", torch.float32, 1)
    sizes = _dev(group_sizes, "group_sizes", torch.int32, 1)
    offs = _dev(group_offsets, "group_offsets", torch.int32, 1)
    padded = _dev(group_padded_offsets, "group_padded_offsets", torch.int32, 1)
    gidx = _dev(group_idx_for_bx, "group_idx_for_bx", torch.int32, 1)
    ul = _dev(up_logits, "up_logits", torch.float16, 2)
    o = _dev(out, "out", torch.float16, 2)
    rows, H = x.shape
    E, I, H2 = g.shape
    if H2 != H or tuple(u.shape) != (E, I, H) or tuple(d.shape) != (E, H, I):
        raise ValueError("weight shapes do not match [E, I, H] / [E, H, I]")
    if tuple(ul.shape) != (rows, I) or tuple(o.shape) != (rows, H):
        raise ValueError("up_logits / out shapes do not match the padded rows")
    if sizes.numel() != E or offs.numel() < E or padded.numel() < E:
        raise ValueError("table lengths do not match n_experts")
    args = (_ptr(x), rows, H, _ptr(g), _ptr(u), _ptr(d), E, I, _ptr(rw), rw.numel(),
            _ptr(sizes), _ptr(offs), _ptr(padded), _ptr(gidx), gidx.numel(),
            _ptr(ul), _ptr(o), _ptr(status), _stream(stream))
    if single_launch_workspace is not None:
        ws = single_launch_workspace
        _check(lib().moe_fused_forward_single_launch(*args[:17], _ptr(ws), ws.numel() * ws.element_size(),
                                                     *args[17:]), "moe_fused_forward_single_launch")
    elif flags == (MOE_RUN_PHASE1 | MOE_RUN_PHASE2):
        _check(lib().moe_fused_forward(*args), "moe_fused_forward")
    else:
        _check(lib().moe_fused_forward_ex(*args, int(flags)), "moe_fused_forward_ex")
    return o


def fused_forward_static_workspace(stacked_expert_tokens, gate_w, up_w, down_w,
                                   routed_expert_weights, group_sizes, group_offsets,
                                   group_padded_offsets, group_idx_for_bx, out,
                                   status=None, stream=None):
    """The fused forward without an up_logits argument, for callers that
    cannot allocate device memory: the workspace is the library's fixed
    64 MiB array (total_padded_tokens * intermediate * 2 bytes at most).
    Calls share that array, so calls that overlap on the GPU race."""
    import torch
    x = _dev(stacked_expert_tokens, "stacked_expert_tokens", torch.float16, 2)
    g = _dev(gate_w, "gate_w", torch.float16, 3)
    u = _dev(up_w, "up_w", torch.float16, 3)
    d = _dev(down_w, "down_w", torch.float16, 3)
    rw = _dev(routed_expert_weights, "routed_expert_weights", torch.float32, 1)
    tabs = [_dev(t, n, torch.int32, 1) for t, n in
            ((group_sizes, "group_sizes"), (group_offsets, "group_offsets"),
             (group_padded_offsets, "group_padded_offsets"), (group_idx_for_bx, "group_idx_for_bx"))]
    o = _dev(out, "out", torch.float16, 2)
    rows, H = x.shape
    E, I, _ = g.shape
    if tuple(o.shape) != (rows, H):
        raise ValueError("out shape does not match the padded rows")
    st = lib().moe_fused_forward_static_workspace(
        _ptr(x), rows, H, _ptr(g), _ptr(u), _ptr(d), E, I, _ptr(rw), rw.numel(),
        *[_ptr(t) for t in tabs], tabs[3].numel(), _ptr(o), _ptr(status), _stream(stream))
    _check(st, "moe_fused_forward_static_workspace")
    return o


def pack_routed(topk_ids, topk_weights, x_tokens, tables, rows_total: int | None = None,
                stacked=None, routed_weights=None, pair_rows=None, workspace=None,
                status=None, stream=None) -> dict:
    """Grouped, padded activations, compact routed weights and every pair's
    padded row, from token-major inputs (all device tensors).  Preallocated
    outputs may be passed; padding rows of ``stacked`` are left untouched
    (a new ``stacked`` is filled with fp16 NaN there)."""
    import torch
    ids = _dev(topk_ids, "topk_ids", torch.int32, 2)
    T, k = ids.shape
    E = tables["group_sizes"].numel()
    x = _dev(x_tokens, "x_tokens", torch.float16, 2) if x_tokens is not None else None
    tw = _dev(topk_weights, "topk_weights", torch.float32, 2) if topk_weights is not None else None
    H = x.shape[1] if x is not None else 128
    if rows_total is None:
        rows_total = tables["group_idx_for_bx"].numel() * BLOCK_TOKEN
    dev = ids.device
    if stacked is None and x is not None:
        stacked = torch.full((rows_total, H), float("nan"), dtype=torch.float16, device=dev)
        _used_on(stream, stacked)
    if routed_weights is None and tw is not None:
        routed_weights = torch.empty(T * k, dtype=torch.float32, device=dev)
        _used_on(stream, routed_weights)
    if pair_rows is None:
        pair_rows = torch.empty((T, k), dtype=torch.int32, device=dev)
        _used_on(stream, pair_rows)
    need = int(lib().moe_pack_workspace_bytes(T * k, E))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        _used_on(stream, workspace)
    st = lib().moe_pack_routed(
        _ptr(ids), _ptr(tw), T, k, E, _ptr(x), H, _ptr(tables["group_offsets"]),
        _ptr(tables["group_padded_offsets"]), rows_total, _ptr(stacked), _ptr(routed_weights),
        _ptr(pair_rows), _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream))
    _check(st, "moe_pack_routed")
    return {"stacked_expert_tokens": stacked, "routed_expert_weights": routed_weights,
            "pair_padded_rows": pair_rows}


def combine_routed(out, pair_rows, y=None, stream=None):
    """y[t] = fp16(sum_j out[pair_rows[t, j]]) with an fp32 sum in j order."""
    import torch
    o = _dev(out, "out", torch.float16, 2)
    pr = _dev(pair_rows, "pair_rows", torch.int32, 2)
    T, k = pr.shape
    if y is None:
        y = torch.empty((T, o.shape[1]), dtype=torch.float16, device=o.device)
        _used_on(stream, y)
    st = lib().moe_combine_routed(_ptr(o), o.shape[0], o.shape[1], _ptr(pr), T, k, _ptr(y),
                                  _stream(stream))
    _check(st, "moe_combine_routed")
    return y


def router_topk(x_tokens, router_w, top_k: int, topk_ids=None, topk_weights=None,
                status=None, stream=None, logits=None):
    """Router logits (x·W_gᵀ), softmax over all experts, top-k: returns
    (topk_ids int32 [T, k], topk_weights fp32 [T, k]).  ``logits`` (fp32 [T, n_experts])
    receives the logits, which router_balance and router_backward read."""
    import torch
    x = _dev(x_tokens, "x_tokens", torch.float16, 2)
    w = _dev(router_w, "router_w", torch.float16, 2)
    T, H = x.shape
    E = w.shape[0]
    if w.shape[1] != H:
        raise ValueError("router_w must be [n_experts, hidden]")
    if topk_ids is None:
        topk_ids = torch.empty((T, top_k), dtype=torch.int32, device=x.device)
        _used_on(stream, topk_ids)
    if topk_weights is None:
        topk_weights = torch.empty((T, top_k), dtype=torch.float32, device=x.device)
        _used_on(stream, topk_weights)
    if logits is not None:
        _shaped(logits, "logits", torch.float32, (T, E))
        _check(lib().moe_router_topk_logits(_ptr(x), T, H, _ptr(w), E, int(top_k), _ptr(topk_ids), _ptr(topk_weights),
                                            _ptr(logits), _ptr(status), _stream(stream)), "moe_router_topk_logits")
        return topk_ids, topk_weights
    st = lib().moe_router_topk(_ptr(x), T, H, _ptr(w), E, int(top_k), _ptr(topk_ids),
                               _ptr(topk_weights), _ptr(status), _stream(stream))
    _check(st, "moe_router_topk")
    return topk_ids, topk_weights


_WORKSPACE = {}


def run_kernel(stacked_expert_tokens, gate_w, up_w, down_w, routed_expert_weights,
               group_sizes, group_offsets, group_padded_offsets, group_idx_for_bx, out):
    """The page's submission signature: ``up_logits`` comes from a per-device,
    per-shape workspace cache (allocated once by PyTorch); ``out`` is written in
    place; no synchronisation, no new tensor."""
    import torch
    key = (stacked_expert_tokens.device.index, int(stacked_expert_tokens.shape[0]),
           int(gate_w.shape[1]))
    ws = _WORKSPACE.get(key)
    if ws is None:
        ws = torch.empty((key[1], key[2]), dtype=torch.float16, device=stacked_expert_tokens.device)
        _WORKSPACE[key] = ws
    fused_forward(stacked_expert_tokens, gate_w, up_w, down_w, routed_expert_weights,
                  group_sizes, group_offsets, group_padded_offsets, group_idx_for_bx, ws, out)


_CODES = {}


def _dtype_code(t, name, f32=False):
    """MOE_DTYPE_* of a torch type."""
    if not _CODES:
        import torch
        _CODES.update({torch.float16: MOE_DTYPE_F16, torch.bfloat16: MOE_DTYPE_BF16, torch.float32: MOE_DTYPE_F32})
    code = _CODES.get(t)
    if code is None or (code == MOE_DTYPE_F32 and not f32):
        raise TypeError(f"{name} must be float16{', bfloat16 or float32' if f32 else ' or bfloat16'}, got {t}")
    return code


def _shaped(t, name, dtype, shape):
    """A device tensor of this type and shape."""
    # the common case in one expression; what follows names what is wrong
    if (getattr(t, "is_cuda", False) and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        return t
    t = _dev(t, name, dtype, len(shape))
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _ffn_sizes(x, gate_w, up_w, down_w):
    """The block's type code and sizes, with every array checked."""
    dt = getattr(x, "dtype", None)
    code = _dtype_code(dt, "x")
    # the common case in one expression; the checks below name what is wrong
    if x.is_cuda and x.dim() == 2 and x.is_contiguous() and getattr(gate_w, "is_cuda", False) and gate_w.dim() == 2:
        T, H = x.shape
        I = gate_w.shape[0]
        if (gate_w.dtype is dt and gate_w.shape == (I, H) and gate_w.is_contiguous()
                and getattr(up_w, "is_cuda", False) and up_w.dtype is dt and up_w.shape == (I, H)
                and up_w.is_contiguous() and getattr(down_w, "is_cuda", False) and down_w.dtype is dt
                and down_w.shape == (H, I) and down_w.is_contiguous()):
            return code, dt, T, H, I
    T, H = _dev(x, "x", dt, 2).shape
    I = _dev(gate_w, "gate_w", dt, 2).shape[0]
    _shaped(gate_w, "gate_w", dt, (I, H))
    _shaped(up_w, "up_w", dt, (I, H))
    _shaped(down_w, "down_w", dt, (H, I))
    return code, dt, T, H, I


def gated_ffn(x, gate_w, up_w, down_w, out=None, up_logits=None, gate=None, up=None, status=None, stream=None):
    """The dense gated feed-forward block: ``out = (silu(x·gate_wᵀ) ⊙ (x·up_wᵀ))·down_wᵀ``.

    x [T, hidden], gate_w / up_w [intermediate, hidden], down_w [hidden,
    intermediate], all float16 or all bfloat16; any T, hidden and intermediate
    multiples of 8, contiguous.  ``out`` [T, hidden] and ``up_logits`` [T,
    intermediate] (the gated product, rounded) may be supplied.  For gradients supply
    ``gate`` and ``up`` [T, intermediate] too: they receive the rounded projections, which
    gated_ffn_backward reads with ``up_logits``.  No autograd graph is recorded:
    inputs that require grad are refused while gradients are being recorded."""
    import torch
    code, dt, T, H, I = _ffn_sizes(x, gate_w, up_w, down_w)
    if ((x.requires_grad or gate_w.requires_grad or up_w.requires_grad or down_w.requires_grad)
            and torch.is_grad_enabled()):
        raise RuntimeError("gated_ffn records no autograd graph, but an input requires grad: call it under "
                           "torch.no_grad() and take the gradients from gated_ffn_backward")
    if gate is not None or up is not None:
        if gate is None or up is None:
            raise ValueError("gate and up are stored together: supply both or neither")
        _shaped(gate, "gate", dt, (T, I))
        _shaped(up, "up", dt, (T, I))
    if up_logits is None:
        up_logits = torch.empty((T, I), dtype=dt, device=x.device)
        _used_on(stream, up_logits)
    else:
        _shaped(up_logits, "up_logits", dt, (T, I))
    if out is None:
        out = torch.empty_like(x)
        _used_on(stream, out)
    else:
        _shaped(out, "out", dt, (T, H))
    st = lib().moe_ffn_forward(code, x.data_ptr(), T, H, gate_w.data_ptr(), up_w.data_ptr(), down_w.data_ptr(), I,
                               _ptr(gate), _ptr(up), up_logits.data_ptr(), out.data_ptr(), _status(status),
                               _stream(stream))
    _check(st, "moe_ffn_forward")
    return out


def gated_ffn_backward(d_out, x, gate_w, up_w, down_w, gate, up, up_logits, d_x=None, d_gate_w=None, d_up_w=None,
                       d_down_w=None, workspace=None, status=None, stream=None):
    """Gradients of gated_ffn from d_out [T, hidden] and what the forward stored
    (``gate``, ``up``, ``up_logits``): returns (d_x, d_gate_w, d_up_w, d_down_w) in
    the inputs' type and shapes.  Supplied buffers are written, not added to.
    ``workspace``: a device tensor of at least ffn_backward_workspace_bytes(T,
    intermediate) bytes."""
    import torch
    code, dt, T, H, I = _ffn_sizes(x, gate_w, up_w, down_w)
    _shaped(d_out, "d_out", dt, (T, H))
    for t, name in ((gate, "gate"), (up, "up"), (up_logits, "up_logits")):
        _shaped(t, name, dt, (T, I))
    grads = []
    for t, name, like in ((d_x, "d_x", x), (d_gate_w, "d_gate_w", gate_w), (d_up_w, "d_up_w", up_w),
                          (d_down_w, "d_down_w", down_w)):
        if t is None:
            t = torch.empty_like(like)
            _used_on(stream, t)
        else:
            _shaped(t, name, dt, like.shape)
        grads.append(t)
    if workspace is None:
        workspace = torch.empty(max(ffn_backward_workspace_bytes(T, I), 16), dtype=torch.uint8, device=x.device)
        _used_on(stream, workspace)
    else:
        _dev(workspace, "workspace", getattr(workspace, "dtype", None))
    _check(lib().moe_ffn_backward(code, d_out.data_ptr(), x.data_ptr(), T, H, gate_w.data_ptr(), up_w.data_ptr(),
                                  down_w.data_ptr(), I, gate.data_ptr(), up.data_ptr(), up_logits.data_ptr(),
                                  workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  *[g.data_ptr() for g in grads], _status(status), _stream(stream)), "moe_ffn_backward")
    return tuple(grads)


def ffn_backward_workspace_bytes(n_tokens: int, intermediate: int) -> int:
    return int(lib().moe_ffn_backward_workspace_bytes(int(n_tokens), int(intermediate)))


def _mx4_scale_shape(rows, cols):
    return ((rows + 127) >> 7, cols >> 7, 32, 4, 4)


def _mx4(codes, scales, name, ndim=None):
    """Checked codes and scales of a 4-bit array: its leading sizes and its columns."""
    import torch
    u8 = torch.uint8
    shape = _dev(codes, name, u8, ndim).shape
    if not shape:
        raise ValueError(f"{name} must have a dim of columns")
    cols = 2 * shape[-1]
    rows = shape[0] if len(shape) == 2 else codes.numel() // max(shape[-1], 1)
    if cols == 0 or cols % 128:
        raise ValueError(f"{name} must hold a multiple of 128 columns, got {cols}")
    tiles = _dev(scales, f"{name}_scales", u8).shape
    # row-major scales can be as many bytes: the tiles' own dims tell them apart
    if tiles[-4:] != (cols >> 7, 32, 4, 4) or scales.numel() != ((rows + 127) >> 7) * (cols >> 7) * 512:
        raise ValueError(f"{name}_scales must hold the tiles {_mx4_scale_shape(rows, cols)}, got {tuple(scales.shape)}")
    return (*shape[:-1], cols)


def mx4_quantize(x, src_rows=None, dest_rows=None, n_dest=None, codes=None, scales=None, status=None, stream=None):
    """4-bit microscaled form of x ([rows, cols], or a weight stack [experts, n,
    cols]), float16, bfloat16 or float32, cols a multiple of 128: returns
    (codes uint8 [..., cols/2], scales uint8 [ceil(rows/128), cols/128, 32, 4, 4]),
    the scale of row r, block b at [r//128, b//4, r%32, r//32%4, b%4].

    For a 2-D x, ``src_rows`` [n] int32 picks the rows to convert and ``dest_rows``
    [n] or [n, copies] int32 the rows of a result of ``n_dest`` rows (those of
    ``codes``, where given) that each goes to (negative entries are skipped; result rows not named keep what the given
    ``codes`` and ``scales`` held, and are undefined in new ones).  With
    dest_rows = pack_routed's pair_padded_rows the tokens land in the grouped,
    padded layout."""
    import torch
    dt = getattr(x, "dtype", None)
    code = _dtype_code(dt, "x", f32=True)
    shape = _dev(x, "x", dt).shape
    lists = src_rows is not None or dest_rows is not None
    if len(shape) != 2 and (len(shape) != 3 or lists):
        raise ValueError("x must have 2 dims, or 3 without row lists")
    cols = shape[-1]
    if cols == 0 or cols % 128:
        raise ValueError(f"x must have a multiple of 128 columns, got {cols}")
    n = n_src = n_out = shape[0] if len(shape) == 2 else shape[0] * shape[1]
    copies, lead = 1, shape[:-1]
    if n_dest is not None and dest_rows is None:
        raise ValueError("n_dest goes with dest_rows: without it the result has the converted rows")
    if lists:
        if src_rows is not None:
            n = _dev(src_rows, "src_rows", torch.int32, 1).numel()
        if dest_rows is not None:
            d = _dev(dest_rows, "dest_rows", torch.int32)
            if d.dim() not in (1, 2) or d.shape[0] != n:
                raise ValueError("dest_rows must be [rows converted] or [rows converted, copies]")
            copies = d.shape[1] if d.dim() == 2 else 1
            if n_dest is None:
                if codes is None:
                    raise ValueError("dest_rows needs n_dest (or codes and scales to write)")
                n_dest = _dev(codes, "codes", torch.uint8, 2).shape[0]
            n_out = int(n_dest)
            if n_out < 0:
                raise ValueError(f"n_dest must not be negative, got {n_out}")
        else:
            n_out = n
        lead = (n_out,)
    if codes is None:
        codes = torch.empty((*lead, cols >> 1), dtype=torch.uint8, device=x.device)
        _used_on(stream, codes)
    else:
        _shaped(codes, "codes", torch.uint8, (*lead, cols >> 1))
    if scales is None:
        scales = torch.empty(_mx4_scale_shape(n_out, cols), dtype=torch.uint8, device=x.device)
        _used_on(stream, scales)
    else:
        _shaped(scales, "scales", torch.uint8, _mx4_scale_shape(n_out, cols))
    if copies == 0:
        return codes, scales
    st = lib().moe_mx4_quantize(code, x.data_ptr(), n_src, cols, _ptr(src_rows), n, _ptr(dest_rows), copies, n_out,
                                codes.data_ptr(), scales.data_ptr(), _status(status), _stream(stream))
    _check(st, "moe_mx4_quantize")
    return codes, scales


def mx4_dequantize(codes, scales, dtype, out=None, stream=None):
    """The values that 4-bit codes [..., cols/2] and their scales stand for, in
    ``dtype`` (float16, bfloat16 or float32): [..., cols]."""
    import torch
    code = _dtype_code(dtype, "dtype", f32=True)
    shape = _mx4(codes, scales, "codes")
    cols = shape[-1]
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=codes.device)
        _used_on(stream, out)
    else:
        _shaped(out, "out", dtype, shape)
    rows = shape[0] if len(shape) == 2 else out.numel() // cols
    st = lib().moe_mx4_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, code, out.data_ptr(),
                                  _stream(stream))
    _check(st, "moe_mx4_dequantize")
    return out


def mx4_matmul(a, a_scales, b, b_scales, out=None, dtype=None, status=None, stream=None):
    """out = a·bᵀ of 4-bit a [rows, k] and b [n, k] (codes and scales), fp32 sums,
    float16 or bfloat16 result [rows, n] (``dtype``, float16 unless ``out`` says)."""
    import torch
    rows, k = _mx4(a, a_scales, "a", 2)
    n, kb = _mx4(b, b_scales, "b", 2)
    if kb != k:
        raise ValueError(f"a and b must have the same columns, got {k} and {kb}")
    if out is None:
        out = torch.empty((rows, n), dtype=dtype or torch.float16, device=a.device)
        _used_on(stream, out)
    code = _dtype_code(getattr(out, "dtype", None), "out")
    _shaped(out, "out", out.dtype, (rows, n))
    _check(lib().moe_mx4_matmul(_ptr(a), _ptr(a_scales), rows, k, _ptr(b), _ptr(b_scales), n, code, _ptr(out),
                                _status(status), _stream(stream)), "moe_mx4_matmul")
    return out


def _mx4_tables(group_sizes, group_padded_offsets, group_idx_for_bx, n_experts):
    import torch
    s = _dev(group_sizes, "group_sizes", torch.int32, 1)
    p = _dev(group_padded_offsets, "group_padded_offsets", torch.int32, 1)
    g = _dev(group_idx_for_bx, "group_idx_for_bx", torch.int32, 1)
    if s.numel() != n_experts or p.numel() < n_experts:
        raise ValueError("table lengths do not match n_experts")
    return g.numel()


def mx4_gate_up(x, x_scales, gate, gate_scales, up, up_scales, group_sizes, group_padded_offsets, group_idx_for_bx,
                up_logits, status=None, stream=None):
    """First half of the routed experts with 4-bit operands: x [padded rows, hidden],
    gate / up [experts, intermediate, hidden] (codes and scales).  Writes ``up_logits``
    [padded rows, intermediate] (float16 or bfloat16) on valid rows and returns it."""
    rows, H = _mx4(x, x_scales, "x", 2)
    E, I, Hg = _mx4(gate, gate_scales, "gate", 3)
    if Hg != H or _mx4(up, up_scales, "up", 3) != (E, I, H):
        raise ValueError("weight shapes do not match [E, I, H]")
    code = _dtype_code(getattr(up_logits, "dtype", None), "up_logits")
    _shaped(up_logits, "up_logits", up_logits.dtype, (rows, I))
    m = _mx4_tables(group_sizes, group_padded_offsets, group_idx_for_bx, E)
    _check(lib().moe_mx4_gate_up(_ptr(x), _ptr(x_scales), rows, H, _ptr(gate), _ptr(gate_scales), _ptr(up),
                                 _ptr(up_scales), E, I, _ptr(group_sizes), _ptr(group_padded_offsets),
                                 _ptr(group_idx_for_bx), m, code, _ptr(up_logits), _status(status), _stream(stream)),
           "moe_mx4_gate_up")
    return up_logits


def mx4_down(h, h_scales, down, down_scales, routed_expert_weights, group_sizes, group_offsets,
             group_padded_offsets, group_idx_for_bx, out, status=None, stream=None):
    """Second half of the routed experts with 4-bit operands: h [padded rows,
    intermediate], down [experts, hidden, intermediate] (codes and scales).  Writes
    ``out`` [padded rows, hidden] (float16 or bfloat16), each valid row times its routed
    weight, and returns it."""
    import torch
    rows, I = _mx4(h, h_scales, "h", 2)
    E, H, Id = _mx4(down, down_scales, "down", 3)
    if Id != I:
        raise ValueError("weight shapes do not match [E, H, I]")
    w = _dev(routed_expert_weights, "routed_expert_weights", torch.float32, 1)
    offs = _dev(group_offsets, "group_offsets", torch.int32, 1)
    code = _dtype_code(getattr(out, "dtype", None), "out")
    _shaped(out, "out", out.dtype, (rows, H))
    m = _mx4_tables(group_sizes, group_padded_offsets, group_idx_for_bx, E)
    if offs.numel() < E:
        raise ValueError("table lengths do not match n_experts")
    _check(lib().moe_mx4_down(_ptr(h), _ptr(h_scales), rows, I, _ptr(down), _ptr(down_scales), E, H, _ptr(w), w.numel(),
                              _ptr(group_sizes), _ptr(offs), _ptr(group_padded_offsets), _ptr(group_idx_for_bx), m,
                              code, _ptr(out), _status(status), _stream(stream)), "moe_mx4_down")
    return out


def _placed(t, name, dtype, shape, d):
    """A tensor of this type and shape on the current device ``d``, where the kernels run."""
    # the common case in one expression; what follows names what is wrong
    try:
        if t.get_device() == d and t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return t
    except AttributeError:
        pass
    _shaped(t, name, dtype, shape)
    if t.device.index != d:
        raise ValueError(f"tensors must be on the current device, cuda:{d}; {name} is on {t.device}")
    return t


def _current(stream):
    """The current device and the handle of the stream to use."""
    import torch
    d = torch.cuda.current_device()
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return d, raw(d)
    return d, _stream(stream)


def _routing(logits, topk_ids, token_mask, seq_offsets, d):
    """Checked sizes (T, E, k, sequences) of what the router's losses and gradients read."""
    import torch
    f32, i32 = torch.float32, torch.int32
    if getattr(logits, "dtype", None) is not f32 or logits.dim() != 2:
        _dev(logits, "logits", f32, 2)
    if getattr(topk_ids, "dtype", None) is not i32 or topk_ids.dim() != 2:
        _dev(topk_ids, "topk_ids", i32, 2)
    T, E = logits.shape
    n, k = topk_ids.shape
    if n != T:
        raise ValueError(f"topk_ids must have a row per token, {T}, got {n}")
    _placed(logits, "logits", f32, (T, E), d)
    _placed(topk_ids, "topk_ids", i32, (T, k), d)
    if token_mask is not None:
        dt = getattr(token_mask, "dtype", None)
        if dt not in (torch.bool, torch.uint8):
            raise TypeError(f"token_mask must be bool or uint8, got {dt}")
        _placed(token_mask, "token_mask", dt, (T,), d)
    if seq_offsets is None:
        return T, E, k, 1
    n = _dev(seq_offsets, "seq_offsets", i32, 1).numel()
    if n < 2:
        raise ValueError(f"seq_offsets must hold the bounds of a sequence at least, got {n} of them")
    _placed(seq_offsets, "seq_offsets", i32, (n,), d)
    return T, E, k, n - 1


def _new(like, shape, dtype, stream):
    """A tensor for a call's result or workspace."""
    import torch
    t = torch.empty(shape, dtype=dtype, device=like.device)
    if stream is not None:
        _used_on(stream, t)
    return t


def _workspace(t, nbytes, like, d, stream):
    """Address and bytes of a workspace of that many bytes, or of the given one, and the tensor."""
    import torch
    if t is None:
        if nbytes <= 0:
            return 0, 0, None
        t = _new(like, (nbytes,), torch.uint8, stream)
        return t.data_ptr(), nbytes, t
    dt = getattr(t, "dtype", None)
    _dev(t, "workspace", dt)
    _placed(t, "workspace", dt, t.shape, d)
    return t.data_ptr(), t.numel() * t.element_size(), t


def router_balance(logits, topk_ids, token_mask=None, seq_offsets=None, losses=None, counts=None, seq_tokens=None,
                   workspace=None, status=None, stream=None):
    """The router's losses and per-expert counts from its logits [T, E] fp32 and chosen
    experts [T, k] int32 (router_topk's): returns (losses, counts, seq_tokens).

    losses [2] fp32: the balance loss E/(k·T)·Σ_s 1/T_s·Σ_e counts[s, e]·Σ_t p[t, e] and the z loss
    mean(logsumexp(z)²).  counts [S, E] int32: pairs of sequence s at expert e.  seq_tokens
    [S + 1] int32: the tokens that count in each sequence, then in all.
    ``token_mask`` [T] (bool or uint8): tokens with 0 do not count.  ``seq_offsets`` [S + 1]
    int32: packed sequences, each balanced by itself (one of all tokens without);
    tokens in none do not count.  ``workspace``: a device tensor of at least
    router_balance_workspace_bytes(T, E, S) bytes.  No autograd graph is recorded."""
    import torch
    f32, i32 = torch.float32, torch.int32
    d, handle = _current(stream)
    T, E, k, S = _routing(logits, topk_ids, token_mask, seq_offsets, d)
    if logits.requires_grad and torch.is_grad_enabled():
        raise RuntimeError("router_balance records no autograd graph, but logits requires grad: call it under "
                           "torch.no_grad() and take the gradients from router_backward")
    losses = _new(logits, (2,), f32, stream) if losses is None else _placed(losses, "losses", f32, (2,), d)
    counts = _new(logits, (S, E), i32, stream) if counts is None else _placed(counts, "counts", i32, (S, E), d)
    if seq_tokens is None:
        seq_tokens = _new(logits, (S + 1,), i32, stream)
    else:
        _placed(seq_tokens, "seq_tokens", i32, (S + 1,), d)
    L = lib()
    ws, nbytes, workspace = _workspace(workspace, L.moe_router_balance_workspace_bytes(T, E, S), logits, d, stream)
    st = L.moe_router_balance(logits.data_ptr(), topk_ids.data_ptr(), T, E, k, _ptr(token_mask), _ptr(seq_offsets), S,
                              losses.data_ptr(), counts.data_ptr(), seq_tokens.data_ptr(), ws, nbytes, _status(status),
                              handle)
    _check(st, "moe_router_balance")
    return losses, counts, seq_tokens


def router_balance_workspace_bytes(n_tokens: int, n_experts: int, n_seqs: int = 1) -> int:
    return int(lib().moe_router_balance_workspace_bytes(int(n_tokens), int(n_experts), int(n_seqs)))


def router_backward(x_tokens, router_w, logits, topk_ids, d_topk_weights=None, d_losses=None, counts=None,
                    seq_tokens=None, token_mask=None, seq_offsets=None, d_x=None, d_router_w=None, d_logits=None,
                    workspace=None, status=None, stream=None):
    """Gradients of the router from those of its routed weights (``d_topk_weights`` [T, k] fp32) and of
    router_balance's losses (``d_losses`` [2] fp32 on the device, with the ``counts``
    and ``seq_tokens`` it returned), either or both: returns (d_x, d_router_w) in the inputs' type
    and shapes, float16 or bfloat16; hidden a multiple of 8.  ``token_mask`` and
    ``seq_offsets`` as in router_balance: a token that does not count has a gradient of zero.
    ``d_logits`` (fp32 [T, E]) receives the gradients of the logits.  Supplied buffers are
    written, not added to, and overlap no input.  All but the ids, routed gradients, losses, counts and what describes the
    sequences start on 16-byte boundaries.  ``workspace``: a device tensor of at least
    router_backward_workspace_bytes(T, E, hidden) bytes."""
    import torch
    f32, i32 = torch.float32, torch.int32
    d, handle = _current(stream)
    T, E, k, S = _routing(logits, topk_ids, token_mask, seq_offsets, d)
    dt = getattr(x_tokens, "dtype", None)
    code = _dtype_code(dt, "x_tokens")
    n, H = _dev(x_tokens, "x_tokens", dt, 2).shape
    if n != T:
        raise ValueError(f"x_tokens must have a row per token, {T}, got {n}")
    _placed(x_tokens, "x_tokens", dt, (T, H), d)
    _placed(router_w, "router_w", dt, (E, H), d)
    if d_topk_weights is not None:
        _placed(d_topk_weights, "d_topk_weights", f32, (T, k), d)
    if d_losses is not None:
        _placed(d_losses, "d_losses", f32, (2,), d)
        if counts is None or seq_tokens is None:
            raise ValueError("d_losses goes with the counts and seq_tokens that router_balance returned")
    if counts is not None:
        _placed(counts, "counts", i32, (S, E), d)
    if seq_tokens is not None:
        _placed(seq_tokens, "seq_tokens", i32, (S + 1,), d)
    if d_logits is not None:
        _placed(d_logits, "d_logits", f32, (T, E), d)
    d_x = _new(x_tokens, (T, H), dt, stream) if d_x is None else _placed(d_x, "d_x", dt, (T, H), d)
    d_router_w = _new(x_tokens, (E, H), dt, stream) if d_router_w is None else _placed(d_router_w, "d_router_w", dt, (E, H), d)
    L = lib()
    ws, nbytes, workspace = _workspace(workspace, L.moe_router_backward_workspace_bytes(T, E, H), logits, d, stream)
    st = L.moe_router_backward(code, x_tokens.data_ptr(), T, H, router_w.data_ptr(), E, logits.data_ptr(),
                               topk_ids.data_ptr(), k, _ptr(d_topk_weights), _ptr(d_losses), _ptr(counts),
                               _ptr(seq_tokens), _ptr(token_mask), _ptr(seq_offsets), S, ws, nbytes, d_x.data_ptr(),
                               d_router_w.data_ptr(), _ptr(d_logits), _status(status), handle)
    _check(st, "moe_router_backward")
    return d_x, d_router_w


def router_backward_workspace_bytes(n_tokens: int, n_experts: int, hidden: int) -> int:
    return int(lib().moe_router_backward_workspace_bytes(int(n_tokens), int(n_experts), int(hidden)))


def orthogonalize(update, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, out=None,
                  workspace=None, status=None, stream=None):
    """Orthogonalised update: X = update / max(‖update‖, eps), then ``steps`` times X ← a·X + (b·A + c·A²)·X
    with A = X·Xᵀ and a, b, c the ``coefficients``: the singular vectors stay and the
    singular values come near 1.  ``update`` [rows, cols] or a stack [batch, rows, cols] of any sizes,
    float16, bfloat16 or float32 (a gradient, or a momentum); returns bfloat16 of its shape
    (``out`` may be supplied).  Each matrix of a stack is taken by itself; one of zeros stays zeros
    whatever ``eps`` is (a norm is taken as at least that of entries of 1.7e-21).  Products
    are of 16-bit operands with fp32 sums: the result is within 2e-3 to 3e-3 of the exact one, root mean
    square, bf16's own rounding included.  ``out`` does not overlap ``update``, and both start on 16-byte boundaries (a
    matrix of a stack of odd sizes, or a view into a buffer of several, may not: clone it, or pass the stack).
    ``workspace``: a device tensor of at least orthogonalize_workspace_bytes(batch, rows, cols) bytes."""
    import torch
    dt = getattr(update, "dtype", None)
    code = _dtype_code(dt, "update", f32=True)
    shape = _dev(update, "update", dt).shape
    if len(shape) not in (2, 3):
        raise ValueError(f"update must have 2 or 3 dims, got {len(shape)}")
    rows, cols = shape[-2:]
    batch = shape[0] if len(shape) == 3 else 1
    if rows == 0 or cols == 0:
        raise ValueError(f"update must have rows and columns, got {tuple(shape)}")
    if update.requires_grad and torch.is_grad_enabled():
        raise RuntimeError("orthogonalize records no autograd graph, but update requires grad: call it under "
                           "torch.no_grad()")
    a, b, c = coefficients
    d, handle = _current(stream)
    _placed(update, "update", dt, shape, d)
    bf16 = torch.bfloat16
    out = _new(update, shape, bf16, stream) if out is None else _placed(out, "out", bf16, shape, d)
    L = lib()
    ws, nbytes, workspace = _workspace(workspace, L.moe_orthogonalize_workspace_bytes(batch, rows, cols), update, d, stream)
    st = L.moe_orthogonalize(code, update.data_ptr(), batch, rows, cols, int(steps), float(a), float(b), float(c),
                             float(eps), ws, nbytes, out.data_ptr(), _status(status), handle)
    _check(st, "moe_orthogonalize")
    return out


def orthogonalize_workspace_bytes(batch: int, rows: int, cols: int) -> int:
    return int(lib().moe_orthogonalize_workspace_bytes(int(batch), int(rows), int(cols)))
