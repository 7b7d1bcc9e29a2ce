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


def plain_layer(seed=1):
    return ops.LoRALinear(160, 272, 8, 16.0, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("assign", [False, True])
@pytest.mark.parametrize("through_file", [False, True])
def test_a_checkpoint_of_a_quantised_layer_loads_into_a_fresh_one(assign, through_file):
    """Into a layer with a bf16 base and into one in the 8-bit form, alone and
    inside a model."""
    src = quantized_layer(seed=3)
    state = {"0." + k: v for k, v in src.state_dict().items()}
    assert sorted(state) == ["0.lora_A", "0.lora_B", "0.weight_codes", "0.weight_scales"]
    if through_file:
        f = io.BytesIO()
        torch.save(state, f)
        f.seek(0)
        state = torch.load(f, weights_only=True)
    for fresh in (plain_layer(), quantized_layer(seed=4)):
        model = torch.nn.Sequential(fresh)
        result = model.load_state_dict(state, strict=True, assign=assign)
        assert not result.missing_keys and not result.unexpected_keys
        m = model[0]
        assert m.weight is None and "base=e4m3" in repr(m)
        for a, b in zip(raw(m), raw(src)):
            assert torch.equal(a, b)
        assert torch.equal(m.lora_A, src.lora_A) and torch.equal(m.lora_B, src.lora_B)
        assert sorted(m.state_dict()) == sorted(src.state_dict())
        if not assign:
            assert m.weight_codes.data_ptr() != state["0.weight_codes"].data_ptr()


def test_a_checkpoint_fills_a_layer_built_on_meta():
    src = quantized_layer(seed=5)
    m = ops.LoRALinear(160, 272, 8, 16.0, device="meta")
    m.load_state_dict(src.state_dict(), assign=True)
    for a, b in zip(raw(m), raw(src)):
        assert torch.equal(a, b)


def test_other_checkpoints_are_refused_and_leave_the_weight():
    """Codes of another layer's size, codes without scales, and a bf16
    checkpoint for an 8-bit layer."""
    m = plain_layer()
    for state in (quantized_layer(d_in=176).state_dict(), quantized_layer(d_out=16).state_dict(),
                  {k: v for k, v in quantized_layer().state_dict().items() if k != "weight_scales"}):
        with pytest.raises(RuntimeError, match="weight"):
            m.load_state_dict(state)
        assert m.weight is not None and torch.equal(m.weight, plain_layer().weight)
    q = quantized_layer()
    before = [b.clone() for b in raw(q)]
    with pytest.raises(RuntimeError, match="weight_codes"):
        q.load_state_dict(m.state_dict())
    for a, b in zip(raw(q), before):
        assert torch.equal(a, b)


def test_plain_checkpoints_load_as_before():
    src, m = plain_layer(2), plain_layer(3)
    m.load_state_dict(src.state_dict())
    assert torch.equal(m.weight, src.weight) and sorted(m.state_dict()) == ["lora_A", "lora_B", "weight"]


def test_a_layer_pickled_without_dropout_still_runs():
    """Layers pickled whole before the module had a dropout have no such
    attribute."""
    m = plain_layer()
    assert m.__dict__.pop("dropout") == 0.0
    f = io.BytesIO()
    torch.save(m, f)
    f.seek(0)
    m = torch.load(f, weights_only=False)
    with torch._subclasses.fake_tensor.FakeTensorMode(allow_non_fake_inputs=True):
        x = torch.empty(3, 160, dtype=torch.bfloat16)
        assert m(x).shape == (3, 272) and m.eval()(x).shape == (3, 272)
    assert "dropout" not in repr(m)


def test_dropout_that_would_drop_everything_is_refused_at_once():
    """p is held as round(65536 p) / 65536: from 1 - 2^-17 on that is 1, which
    the library refuses at every call."""
    for p in (1.0 - 2.0 ** -17, 0.999999, 1.0 - 2.0 ** -30, 1.0):
        with pytest.raises(ValueError, match="dropout"):
            ops.LoRALinear(16, 16, 8, 8.0, dropout=p)
    for p in (0.0, 1e-9, 1.0 - 2.0 ** -16, 1.0 - 2.0 ** -17 - 2.0 ** -23):
        assert ops.LoRALinear(16, 16, 8, 8.0, dropout=p).dropout == p
    with torch.device("meta"):
        assert ops.LoRALinear(16, 16, 8, 8.0, dropout=0.1).lora_A.is_meta


def test_the_refusal_of_p_names_the_rounding(built_lib):
    assert "65536" in built_lib.lora_status_string(11)
