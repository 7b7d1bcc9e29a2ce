"""The operators with dropout and with an 8-bit base on CPU: fake shapes,
autograd wiring, a trace without graph breaks, the module's options."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from lora_linear_layer_b200 import ops

BF16 = torch.bfloat16


def _inputs(device, fp8, M=32, d_in=64, d_out=48, r=8):
    e = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device=device)
    W = e(d_out, d_in, dtype=torch.float8_e4m3fn if fp8 else BF16)
    Ws = e((d_out + 127) // 128, (d_in + 127) // 128, dtype=torch.float8_e8m0fnu) if fp8 else None
    return e(M, d_in), W, Ws, e(r, d_in), e(d_out, r)


@pytest.mark.parametrize("fp8", [False, True])
def test_fake_shapes(fp8):
    with FakeTensorMode():
        X, W, Ws, A, B = _inputs("cuda", fp8)
        rng = torch.empty(2, dtype=torch.int64, device="cuda")
        Y, saved = torch.ops.lora_b200.lora_linear_adapter(X, W, Ws, A, B, 2.0, 0.1, rng)
        assert Y.shape == (32, 48) and Y.dtype == BF16 and saved.dtype == torch.uint8
        assert saved.numel() == 32 * 16 * 2
        assert torch.ops.lora_b200.lora_linear_adapter(X, W, Ws, A, B, 2.0, 0.1, rng, False)[1].numel() == 0
        for f32 in (False, True):
            dX, dA, dB = torch.ops.lora_b200.lora_linear_adapter_bwd(X, W, Ws, A, B, Y, saved, 2.0, 0.1, rng, f32)
            assert dX.shape == X.shape and dA.shape == A.shape and dB.shape == B.shape
            assert dA.dtype == dB.dtype == (torch.float32 if f32 else BF16)


@pytest.mark.parametrize("fp8", [False, True])
def test_autograd_reaches_x_a_and_b(fp8):
    X, W, Ws, A, B = _inputs("meta", fp8)
    for t in (X, A, B):
        t.requires_grad_(True)
    rng = torch.empty(2, dtype=torch.int64, device="meta")
    Y, _ = torch.ops.lora_b200.lora_linear_adapter(X, W, Ws, A, B, 2.0, 0.1, rng)
    for g, t in zip(torch.autograd.grad(Y.sum(), (X, A, B)), (X, A, B)):
        assert g.shape == t.shape


def test_refusals():
    with FakeTensorMode():
        X, W, Ws, A, B = _inputs("cuda", False)
        with pytest.raises(ValueError, match="rng"):
            torch.ops.lora_b200.lora_linear_adapter(X, W, None, A, B, 2.0, 0.1, None)
        with pytest.raises(ValueError):
            torch.ops.lora_b200.lora_linear_adapter(X, W, None, A[:, :32], B, 2.0, 0.0, None)
        W.requires_grad_(True)
        X.requires_grad_(True)
        with pytest.raises(RuntimeError, match="frozen"):
            torch.ops.lora_b200.lora_linear_adapter(X, W, None, A, B, 2.0, 0.0, None)
    for p in (-0.1, 1.0, float("nan")):
        with pytest.raises(ValueError, match="dropout"):
            ops.LoRALinear(16, 16, 8, 8.0, dropout=p)


@pytest.mark.parametrize("d_in, d_out", [(64, 24), (24, 64)])
def test_quantize_base_refuses_sizes_that_the_8_bit_layer_does_not_have(d_in, d_out):
    m = ops.LoRALinear(d_in, d_out, 8, 8.0)
    with pytest.raises(ValueError, match="multiples of 16"):
        m.quantize_base()
    assert m.weight is not None and "weight_codes" not in m.state_dict()


@pytest.mark.parametrize("train", [True, False])
def test_module_traces_without_a_graph_break(train):
    with FakeTensorMode():
        m = ops.LoRALinear(64, 48, 8, 16.0, device="cuda", dropout=0.1).train(train)
        x = torch.empty(4, 8, 64, dtype=BF16, device="cuda", requires_grad=True)
        y = m(x)
        assert y.shape == (4, 8, 48) and y.requires_grad


def test_saved_bytes_are_the_librarys(built_lib):
    for M, r in ((1, 8), (5, 16), (300, 24), (4096, 128)):
        assert 2 * ops._saved_bytes(M, r) == built_lib.lora_bwd_workspace_size(M, 64, 64, r)
        assert built_lib.lora_fp8_workspace_size(M, 64, 64, r) >= ops._saved_bytes(M, r)
