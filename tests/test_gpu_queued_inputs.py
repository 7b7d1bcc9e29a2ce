"""Calls queued one behind another, each of which reads what the one before it
has just written: the results of the same calls with a wait after every one,
bit for bit.  (Every launch is programmatic, so a kernel that read its inputs
before its wait would read the old ones.)"""
import pytest
import torch

from test_gpu_adapter_dropout import BF16, make, rng_tensor

pytestmark = pytest.mark.gpu

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.mark.parametrize("d_out,d_in", [(256, 128), (1024, 2560), (4096, 4096)])
def test_conversions_read_what_was_just_written(gpu, d_out, d_in):
    """Copy, quantise and dequantise in one set of buffers, for one weight
    after another."""
    L, steps = gpu, 10
    g = torch.Generator(device="cuda").manual_seed(d_out)
    new = [(torch.randn(d_out, d_in, generator=g, device="cuda") * 2.0 ** (i - 5)).to(BF16) for i in range(steps)]

    def run(wait):
        W = torch.full((d_out, d_in), 3.0, dtype=BF16, device="cuda")
        Wq = torch.full((d_out, d_in), 77, dtype=torch.uint8, device="cuda").view(E4M3)
        Ws = torch.full(((d_out + 127) // 128, (d_in + 127) // 128), 77, dtype=torch.uint8, device="cuda").view(E8M0)
        out = [torch.zeros(d_out, d_in, dtype=BF16, device="cuda") for _ in range(steps)]
        torch.cuda.synchronize()
        for source, o in zip(new, out):
            for call, args in ((L.lora_restore, (source, W)), (L.lora_quantize_fp8, (W, Wq, Ws)),
                               (L.lora_dequantize_fp8, (Wq, Ws, o)), (L.lora_restore, (o, W)),
                               (L.lora_quantize_fp8, (W, Wq, Ws)), (L.lora_dequantize_fp8, (Wq, Ws, o))):
                call(*args)
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return out

    want = run(True)
    for _ in range(5):
        for o, w in zip(run(False), want):
            assert torch.equal(o, w)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M", [1, 20, 300, 1100])
def test_each_layer_reads_the_one_before(gpu, fp8, M):
    """Forwards in a row, every one's Y the next one's X, in two buffers."""
    L, d, r, layers = gpu, 1024, 16, 24
    t = {k: v.cuda() for k, v in make(M, d, d, r).items()}
    Wq, Ws = torch.empty(d, d, dtype=E4M3, device="cuda"), torch.empty(d // 128, d // 128, dtype=E8M0, device="cuda")
    L.lora_quantize_fp8(t["W"], Wq, Ws)
    rng = rng_tensor(3, 4)
    size = (L.lora_fp8_workspace_size if fp8 else L.lora_bwd_workspace_size)(M, d, d, r)

    def run(wait):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        x, y = t["X"].clone(), torch.zeros_like(t["X"])
        torch.cuda.synchronize()
        for _ in range(layers):
            if fp8:
                L.lora_fwd_fp8(x, Wq, Ws, t["A"], t["B"], y, 2.0, ws, 0.25, rng)
            else:
                L.lora_fwd_dropout(x, t["W"], t["A"], t["B"], y, 2.0, 0.25, rng, ws)
            if wait:
                torch.cuda.synchronize()
            x, y = y, x
        torch.cuda.synchronize()
        return x

    want = run(True)
    assert torch.isfinite(want.float()).all()
    for _ in range(10):
        assert torch.equal(run(False), want)
    assert L.lora_get_device_status() == 0
