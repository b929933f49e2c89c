"""What the binding refuses before it reaches the library, on tensors without data: device
tensors of every shape exist, and nothing is launched."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import routed_grouped_gemm_dispatch_gb300 as moe

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer")


@pytest.fixture
def fake():
    """Tensors made inside have a device, a type, sizes and strides, and no memory."""
    moe.build()
    moe.lib()
    with FakeTensorMode():
        yield lambda *shape, dt=torch.uint8: torch.empty(shape, dtype=dt, device="cuda")


def test_scales_in_another_order_are_refused(fake):
    """Row-major scales, [rows, columns / 32], are as many bytes as the tiles where rows are a
    multiple of 128; so are tiles of another shape."""
    c, t = fake(256, 256), fake(2, 4, 32, 4, 4)
    assert moe._mx4(c, t, "a", 2) == (256, 512)
    assert moe._mx4(fake(2, 128, 256), t, "a", 3) == (2, 128, 512)
    assert moe._mx4(fake(2, 128, 256), fake(2, 1, 4, 32, 4, 4), "a", 3) == (2, 128, 512)     # a stack's tiles apart
    assert moe._mx4(fake(0, 256), fake(0, 4, 32, 4, 4), "a", 2) == (0, 512)
    other = [fake(256, 16), fake(4096), fake(4, 2, 32, 4, 4), fake(2, 4, 4, 32, 4), fake(2, 4, 512), fake(8, 32, 4, 4)]
    w, ws, h = fake(1, 128, 256), fake(1, 4, 32, 4, 4), fake(256, 128, dt=torch.float16)
    i32 = [fake(n, dt=torch.int32) for n in (1, 2, 2, 2)]
    for s in other:
        with pytest.raises(ValueError, match="must hold the tiles"):
            moe.mx4_dequantize(c, s, torch.float16)
        with pytest.raises(ValueError, match="a_scales must hold the tiles"):
            moe.mx4_matmul(c, s, c, t)
        with pytest.raises(ValueError, match="b_scales must hold the tiles"):
            moe.mx4_matmul(c, t, c, s)
        with pytest.raises(ValueError, match="x_scales must hold the tiles"):
            moe.mx4_gate_up(c, s, w, ws, w, ws, i32[0], i32[2], i32[3], h)
        with pytest.raises(ValueError, match="h_scales must hold the tiles"):
            moe.mx4_down(c, s, w, ws, fake(5, dt=torch.float32), *i32, h)
    # a weight stack's
    with pytest.raises(ValueError, match="gate_scales must hold the tiles"):
        moe.mx4_gate_up(c, t, w, fake(128, 16), w, ws, i32[0], i32[2], i32[3], h)
    with pytest.raises(ValueError, match="up_scales must hold the tiles"):
        moe.mx4_gate_up(c, t, w, ws, w, fake(128, 16), i32[0], i32[2], i32[3], h)
    with pytest.raises(ValueError, match="down_scales must hold the tiles"):
        moe.mx4_down(c, t, w, fake(128, 16), fake(5, dt=torch.float32), *i32, h)


def test_n_dest_has_to_agree(fake):
    """n_dest is the rows of the result that dest_rows points into: not another number than the given
    codes have, and nothing without dest_rows."""
    x, dest = fake(4, 256, dt=torch.float16), fake(4, dt=torch.int32)
    codes, scales = fake(20, 128), fake(1, 2, 32, 4, 4)
    for n in (10, 0, 21):
        with pytest.raises(ValueError, match="codes must have shape"):
            moe.mx4_quantize(x, dest_rows=dest, n_dest=n, codes=codes, scales=scales)
    for n in (0, 4, 7):
        with pytest.raises(ValueError, match="n_dest goes with dest_rows"):
            moe.mx4_quantize(x, n_dest=n)
        with pytest.raises(ValueError, match="n_dest goes with dest_rows"):
            moe.mx4_quantize(x, src_rows=dest, n_dest=n)
    with pytest.raises(ValueError, match="n_dest"):
        moe.mx4_quantize(x, dest_rows=dest, n_dest=-1)
    with pytest.raises(ValueError, match="codes must have 2 dims"):
        moe.mx4_quantize(x, dest_rows=dest, codes=fake(2, 20, 128))
    with pytest.raises(TypeError, match="codes"):
        moe.mx4_quantize(x, dest_rows=dest, codes=[1, 2])
    with pytest.raises(ValueError, match="scales must have shape"):
        moe.mx4_quantize(x, dest_rows=dest, n_dest=20, codes=codes, scales=fake(2, 2, 32, 4, 4))


@pytest.mark.parametrize("which", ["x", "gate_w", "up_w", "down_w"])
def test_autograd_is_not_lost_silently(fake, which):
    """gated_ffn records no graph: with an input that asks for gradients it says so, unless none are
    being recorded."""
    dt = torch.bfloat16
    a = {"x": fake(3, 16, dt=dt), "gate_w": fake(24, 16, dt=dt), "up_w": fake(24, 16, dt=dt), "down_w": fake(16, 24, dt=dt)}
    a[which].requires_grad_()
    h = fake(3, 16, dt=dt)                        # a wrong up_logits: refused next, where the call goes on
    with pytest.raises(RuntimeError, match="gated_ffn_backward"):
        moe.gated_ffn(**a, up_logits=h)
    for quiet in (torch.no_grad(), torch.inference_mode()):
        with quiet, pytest.raises(ValueError, match="up_logits"):
            moe.gated_ffn(**a, up_logits=h)
    a[which] = a[which].detach()
    with pytest.raises(ValueError, match="up_logits"):
        moe.gated_ffn(**a, up_logits=h)


def test_status_and_workspace_are_device_memory(fake):
    """The kernels write to both: a status word is one int32 on the device at least, a workspace is there too."""
    dt = torch.float16
    x, w, d, h = fake(3, 16, dt=dt), fake(24, 16, dt=dt), fake(16, 24, dt=dt), fake(3, 24, dt=dt)
    c, s = fake(128, 64), fake(1, 1, 32, 4, 4)
    cw, sw, i32 = fake(1, 128, 64), fake(1, 1, 32, 4, 4), [fake(n, dt=torch.int32) for n in (1, 2, 2, 1)]
    out = fake(128, 128, dt=dt)
    calls = [lambda st: moe.gated_ffn(x, w, w, d, status=st),
             lambda st: moe.gated_ffn_backward(x, x, w, w, d, h, h, h, status=st),
             lambda st: moe.mx4_quantize(fake(3, 128, dt=dt), status=st),
             lambda st: moe.mx4_matmul(c, s, c, s, status=st),
             lambda st: moe.mx4_gate_up(c, s, cw, sw, cw, sw, i32[0], i32[2], i32[3], out, status=st),
             lambda st: moe.mx4_down(c, s, cw, sw, fake(5, dt=torch.float32), *i32, out, status=st)]
    for call in calls:
        with pytest.raises(ValueError, match="status must be a CUDA tensor"):
            call(torch.zeros(1, dtype=torch.int32))
        with pytest.raises(TypeError, match="status must be torch.int32"):
            call(fake(4))
        with pytest.raises(ValueError, match="status must hold"):
            call(fake(0, dt=torch.int32))
        with pytest.raises(TypeError, match="status must be a torch.Tensor"):
            call(0x1000)
    for ws, error, text in ((torch.zeros(1 << 16, dtype=torch.uint8), ValueError, "CUDA"), (0x1000, TypeError, "Tensor"),
                            (fake(1 << 17)[::2], ValueError, "contiguous")):
        with pytest.raises(error, match=f"workspace must be .*{text}"):
            moe.gated_ffn_backward(x, x, w, w, d, h, h, h, workspace=ws)
