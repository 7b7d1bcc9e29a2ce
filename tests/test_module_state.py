"""LoRALinear as a module: casts, checkpoints, pickles (CPU)."""
import copy
import io

import pytest
import torch

from lora_linear_layer_b200 import ops

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def quantized_layer(d_in=160, d_out=272, r=8, seed=0):
    """A layer in the form that quantize_base() leaves it in, with every byte
    but the NaN codes among its codes and scales."""
    m = ops.LoRALinear(d_in, d_out, r, 16.0)
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (d_out, d_in), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 5
    scales = torch.randint(1, 254, ((d_out + 127) // 128, (d_in + 127) // 128), generator=g, dtype=torch.uint8)
    m.weight = None
    m.register_buffer("weight_codes", codes.view(E4M3))
    m.register_buffer("weight_scales", scales.view(E8M0))
    return m


def raw(m):
    assert m.weight_codes.dtype == E4M3 and m.weight_scales.dtype == E8M0
    return m.weight_codes.view(torch.uint8), m.weight_scales.view(torch.uint8)


CASTS = {
    "to(bfloat16)": lambda m: m.to(torch.bfloat16),
    "bfloat16": lambda m: m.bfloat16(),
    "half": lambda m: m.half(),
    "float": lambda m: m.float(),
    "double": lambda m: m.double(),
    "type": lambda m: m.type(torch.float32),
    "to(device, dtype)": lambda m: m.to("cpu", torch.bfloat16),
    "cpu": lambda m: m.cpu(),
    "share_memory": lambda m: m.share_memory(),
    "deepcopy": copy.deepcopy,
    "in a model": lambda m: torch.nn.Sequential(m, torch.nn.Linear(4, 4)).to(torch.bfloat16)[0],
}


@pytest.mark.parametrize("cast", sorted(CASTS))
def test_a_cast_leaves_codes_and_scales(cast):
    m = quantized_layer()
    before = [b.clone() for b in raw(m)]
    m = CASTS[cast](m)
    for a, b in zip(raw(m), before):
        assert torch.equal(a, b)
    assert sorted(n for n, _ in m.named_buffers()) == ["weight_codes", "weight_scales"] and m.weight is None


def test_a_cast_reaches_the_adapter_and_a_plain_weight():
    m = quantized_layer().double()
    assert m.lora_A.dtype == m.lora_B.dtype == torch.float64
    m = ops.LoRALinear(16, 16, 8, 8.0).half()
    assert m.weight.dtype == m.lora_A.dtype == torch.float16


def test_codes_move_to_another_device():
    m = quantized_layer().to("meta")
    assert m.weight_codes.is_meta and m.weight_scales.is_meta
    raw(m)
    m = m.to_empty(device="cpu")
    assert m.weight_codes.device.type == "cpu" and m.weight_codes.shape == (272, 160)
    raw(m)
