"""Refusals of the router's losses and gradients and of the orthogonalised updates: every call here fails a
check on the host, before anything is enqueued."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import routed_grouped_gemm_dispatch_gb300 as moe

NULL, SHAPE, ALIGN, LIMIT, WORKSPACE = -1, -2, -3, -7, -8
pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer")


@pytest.fixture(scope="module")
def L():
    moe.build()
    return moe.lib()


BAL = dict(z=0x1000, ids=0x2000, T=50000, E=24, k=3, mask=0x3000, offs=0x4000, S=4, losses=0x5000, counts=0x6000, tokens=0x7000,
           ws=0x8000, n=1 << 20)


def bal(L, **kw):
    a = {**BAL, **kw}
    return L.moe_router_balance(a["z"], a["ids"], a["T"], a["E"], a["k"], a["mask"], a["offs"], a["S"], a["losses"],
                                a["counts"], a["tokens"], a["ws"], a["n"], None, None)


def sizes(call, L):
    """What both calls that read logits and ids refuse."""
    assert call(L, T=-1) == SHAPE
    assert call(L, E=0) == SHAPE
    assert call(L, k=0) == SHAPE
    assert call(L, k=25) == SHAPE
    assert call(L, S=0) == SHAPE
    assert call(L, offs=None) == SHAPE                 # several sequences and no bounds
    assert call(L, T=(1 << 24) + 1) == LIMIT
    assert call(L, E=1025) == LIMIT
    assert call(L, k=17) == LIMIT
    assert call(L, S=65536) == LIMIT
    assert call(L, ws=None) == WORKSPACE
    assert call(L, ws=0x8008) == ALIGN
    assert call(L, z=0x1004) == ALIGN
    assert call(L, z=None) == NULL
    assert call(L, ids=None) == NULL


def test_balance_refusals(L):
    sizes(bal, L)
    for key in ("losses", "counts", "tokens"):
        assert bal(L, **{key: None}) == NULL
    need = L.moe_router_balance_workspace_bytes(50000, 24, 4)
    assert L.moe_router_balance_workspace_bytes(64, 24, 2) == 0                # needs none
    assert L.moe_router_balance_workspace_bytes(64, 24, 400) > 0 and L.moe_router_balance_workspace_bytes(1 << 20, 24, 1) > 0
    assert need > 0 and bal(L, n=need - 1) == WORKSPACE
    for bad in ((-1, 24, 4), (500, 0, 4), (500, 1025, 4), (500, 24, 0), (500, 24, 65536), ((1 << 24) + 1, 24, 1)):
        assert L.moe_router_balance_workspace_bytes(*bad) == -1


BWD = dict(dtype=0, x=0x1000, T=50, H=72, w=0x2000, E=24, z=0x3000, ids=0x4000, k=3, dw=0x5000, dl=0x6000, counts=0x7000,
           tokens=0x8000, mask=0x9000, offs=0xA000, S=4, ws=0xB000, n=1 << 30, dx=0xC000, dwg=0xD000, dz=0xE000)


def bwd(L, **kw):
    a = {**BWD, **kw}
    return L.moe_router_backward(a["dtype"], a["x"], a["T"], a["H"], a["w"], a["E"], a["z"], a["ids"], a["k"], a["dw"],
                                 a["dl"], a["counts"], a["tokens"], a["mask"], a["offs"], a["S"], a["ws"], a["n"], a["dx"],
                                 a["dwg"], a["dz"], None, None)


def test_backward_refusals(L):
    sizes(bwd, L)
    assert bwd(L, dtype=2) == SHAPE
    assert bwd(L, H=0) == SHAPE
    assert bwd(L, H=60) == SHAPE
    assert bwd(L, H=(1 << 20) + 8) == LIMIT
    for key in ("x", "w", "dx", "dwg", "counts", "tokens"):    # the last two go with d_losses
        assert bwd(L, **{key: None}) == NULL, key
    for key in ("x", "w", "dx", "dwg", "dz", "z"):
        assert bwd(L, **{key: 0x1008}) == ALIGN, key
    need = L.moe_router_backward_workspace_bytes(50, 24, 72)
    assert need > 0 and bwd(L, n=need - 1) == WORKSPACE
    for bad in ((-1, 24, 72), (50, 0, 72), (50, 1025, 72), (50, 24, 0), (50, 24, (1 << 20) + 8)):
        assert L.moe_router_backward_workspace_bytes(*bad) == -1


ORT = dict(dtype=1, u=0x1000, batch=2, rows=33, cols=50, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, ws=0x2000, n=1 << 30,
           out=0x3000)


def ort(L, **kw):
    a = {**ORT, **kw}
    return L.moe_orthogonalize(a["dtype"], a["u"], a["batch"], a["rows"], a["cols"], a["steps"], a["a"], a["b"], a["c"],
                               a["eps"], a["ws"], a["n"], a["out"], None, None)


def test_orthogonalize_refusals(L):
    for kw in (dict(dtype=3), dict(dtype=-1), dict(batch=-1), dict(rows=0), dict(cols=0), dict(steps=0), dict(eps=-1e-9),
               dict(eps=float("nan")), dict(eps=float("inf"))):
        assert ort(L, **kw) == SHAPE, kw
    for kw in (dict(batch=65536), dict(rows=65537), dict(cols=65537), dict(steps=65), dict(a=65.0), dict(b=-65.0),
               dict(c=float("nan")), dict(a=float("inf")), dict(batch=65535, rows=65536, cols=65536)):
        assert ort(L, **kw) == LIMIT, kw
    for key in ("u", "out"):
        assert ort(L, **{key: None}) == NULL
        assert ort(L, **{key: 0x1008}) == ALIGN
    assert ort(L, ws=0x2008) == ALIGN
    assert ort(L, ws=None) == WORKSPACE
    need = L.moe_orthogonalize_workspace_bytes(2, 33, 50)
    assert need > 0 and ort(L, n=need - 1) == WORKSPACE
    assert ort(L, batch=0, u=None, out=None, ws=None, n=0) == 0                  # nothing to do
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (65536, 1, 1), (1, 65537, 1)):
        assert L.moe_orthogonalize_workspace_bytes(*bad) == -1


def test_router_logits_refusals(L):
    def call(logits, T=5):
        return L.moe_router_topk_logits(0x1000, T, 128, 0x2000, 4, 2, 0x3000, 0x4000, logits, None, None)
    assert call(0x5004) == ALIGN
    assert call(None, 0) == 0


@pytest.fixture
def fake(L, monkeypatch):
    """Tensors made inside have a device, a type, sizes and strides, and no memory."""
    monkeypatch.setattr(moe, "_stream", lambda s: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    with FakeTensorMode():
        yield lambda *shape, dt=torch.float32: torch.empty(shape, dtype=dt, device="cuda")


def test_binding_refusals(fake):
    i32, f16, bf = torch.int32, torch.float16, torch.bfloat16
    z, ids = fake(50, 24), fake(50, 3, dt=i32)
    x, w = fake(50, 72, dt=f16), fake(24, 72, dt=f16)
    on_cpu = torch.zeros((50, 24))
    for call in (lambda **k: moe.router_balance(**{"logits": z, "topk_ids": ids, **k}),
                 lambda **k: moe.router_backward(**{"x_tokens": x, "router_w": w, "logits": z, "topk_ids": ids, **k})):
        with pytest.raises(ValueError, match="CUDA"):
            call(logits=on_cpu)
        with pytest.raises(TypeError, match="logits must be torch.float32"):
            call(logits=fake(50, 24, dt=f16))
        with pytest.raises(ValueError, match="contiguous"):
            call(logits=fake(24, 50).t())
        with pytest.raises(TypeError, match="topk_ids must be torch.int32"):
            call(topk_ids=fake(50, 3, dt=torch.int64))
        with pytest.raises(ValueError, match="topk_ids must have a row per token"):
            call(topk_ids=fake(49, 3, dt=i32))
        with pytest.raises(TypeError, match="token_mask must be bool or uint8"):
            call(token_mask=fake(50))
        with pytest.raises(ValueError, match="token_mask must have shape"):
            call(token_mask=fake(51, dt=torch.bool))
        with pytest.raises(ValueError, match="seq_offsets must hold"):
            call(seq_offsets=fake(1, dt=i32))
        with pytest.raises(TypeError, match="seq_offsets must be torch.int32"):
            call(seq_offsets=fake(3, dt=torch.int64))
        with pytest.raises(ValueError, match="status must be a CUDA tensor"):
            call(status=torch.zeros(1, dtype=i32))
        with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
            call(workspace=torch.zeros(1 << 22, dtype=torch.uint8))
        with pytest.raises(moe.MoeError, match="SHAPE"):
            call(topk_ids=fake(50, 0, dt=i32))
    with pytest.raises(ValueError, match="counts must have shape"):
        moe.router_balance(z, ids, seq_offsets=fake(3, dt=i32), counts=fake(1, 24, dt=i32))
    with pytest.raises(ValueError, match="seq_tokens must have shape"):
        moe.router_balance(z, ids, seq_tokens=fake(1, dt=i32))
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        moe.router_backward(fake(50, 72), w, z, ids)
    with pytest.raises(TypeError, match="router_w must be"):
        moe.router_backward(x, fake(24, 72, dt=bf), z, ids)
    with pytest.raises(ValueError, match="router_w must have shape"):
        moe.router_backward(x, fake(25, 72, dt=f16), z, ids)
    with pytest.raises(ValueError, match="x_tokens must have a row per token"):
        moe.router_backward(fake(49, 72, dt=f16), w, z, ids)
    with pytest.raises(ValueError, match="d_losses goes with"):
        moe.router_backward(x, w, z, ids, d_losses=fake(2))
    with pytest.raises(ValueError, match="counts must have shape"):
        moe.router_backward(x, w, z, ids, d_losses=fake(2), counts=fake(2, 24, dt=i32), seq_tokens=fake(2, dt=i32))
    with pytest.raises(ValueError, match="d_topk_weights must have shape"):
        moe.router_backward(x, w, z, ids, fake(50, 2))
    with pytest.raises(ValueError, match="d_logits must have shape"):
        moe.router_backward(x, w, z, ids, d_logits=fake(50, 25))
    with pytest.raises(ValueError, match="logits must have shape"):
        moe.router_topk(fake(50, 128, dt=f16), fake(24, 128, dt=f16), 3, logits=fake(50, 23))
    with pytest.raises(TypeError, match="update must be float16, bfloat16 or float32"):
        moe.orthogonalize(fake(4, 8, dt=torch.float64))
    with pytest.raises(TypeError, match="update must be"):
        moe.orthogonalize(None)
    with pytest.raises(ValueError, match="2 or 3 dims"):
        moe.orthogonalize(fake(8))
    with pytest.raises(ValueError, match="rows and columns"):
        moe.orthogonalize(fake(4, 0))
    with pytest.raises(ValueError, match="contiguous"):
        moe.orthogonalize(fake(8, 4).t())
    with pytest.raises(ValueError, match="CUDA"):
        moe.orthogonalize(on_cpu)
    with pytest.raises(TypeError, match="out must be torch.bfloat16"):
        moe.orthogonalize(fake(4, 8), out=fake(4, 8))
    with pytest.raises(ValueError):
        moe.orthogonalize(fake(4, 8), coefficients=(1.0, 2.0))
    with pytest.raises(moe.MoeError, match="LIMIT"):
        moe.orthogonalize(fake(4, 8), steps=65)
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.orthogonalize(fake(4, 8), steps=0)


class NoLibrary:
    """Takes every call and says that it went well."""

    def __getattr__(self, name):
        return lambda *a: 1 if name.endswith("_bytes") else 0


@pytest.mark.parametrize("name,n", [("router_balance", 4), ("router_backward", 3), ("orthogonalize", 2)])
@pytest.mark.parametrize("given", [False, True])
def test_allocations_are_recorded(name, n, given, monkeypatch):
    """Whatever a call allocates is recorded on the stream that it is given."""
    class Stream:
        cuda_stream = 0x77

    made, recorded, stream = [], [], Stream() if given else None
    monkeypatch.setattr(moe, "lib", lambda lib=NoLibrary(): lib)
    monkeypatch.setattr(moe, "_stream", lambda s: 0 if s is None else s.cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")
        z, ids = torch.empty((4, 8), device="cuda"), torch.empty((4, 2), dtype=torch.int32, device="cuda")
        x, w = torch.empty((4, 16), dtype=torch.float16, device="cuda"), torch.empty((8, 16), dtype=torch.float16, device="cuda")
        args = {"router_balance": (z, ids), "router_backward": (x, w, z, ids), "orthogonalize": (x,)}[name]
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((id(t), s)))
        inside = []
        for owner, f in ((torch, "empty"), (torch, "empty_like")):
            def spy(*a, _f=getattr(owner, f), **k):
                inside.append(1)
                r = _f(*a, **k)
                inside.pop()
                if not inside:
                    made.append(r)
                return r
            monkeypatch.setattr(owner, f, spy)
        getattr(moe, name)(*args, stream=stream)
    assert len(made) == n
    assert recorded == ([(id(t), stream) for t in made] if given else [])


def test_other_devices_are_refused(fake, monkeypatch):
    """The kernels run on the current device, whatever device the tensors are on."""
    z, ids, x, w = fake(4, 8), fake(4, 2, dt=torch.int32), fake(4, 16, dt=torch.float16), fake(8, 16, dt=torch.float16)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: moe.router_balance(z, ids), lambda: moe.router_backward(x, w, z, ids), lambda: moe.orthogonalize(x)):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_autograd_is_not_lost_silently(fake):
    z, ids, u = fake(4, 8).requires_grad_(), fake(4, 2, dt=torch.int32), fake(4, 16).requires_grad_()
    with pytest.raises(RuntimeError, match="router_backward"):
        moe.router_balance(z, ids)
    with pytest.raises(RuntimeError, match="no_grad"):
        moe.orthogonalize(u)
    with torch.no_grad(), pytest.raises(ValueError, match="losses must have shape"):
        moe.router_balance(z, ids, losses=fake(3))
    with torch.no_grad(), pytest.raises(TypeError, match="out must be"):
        moe.orthogonalize(u, out=fake(4, 16))
