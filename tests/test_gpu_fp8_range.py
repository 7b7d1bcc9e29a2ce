"""The 8-bit base over the whole range of its scales, and a quantised layer
after a cast and through a checkpoint."""
import numpy as np
import pytest
import torch

from test_gpu_adapter_dropout import BF16, make
from test_gpu_ops_adapter import layer

pytestmark = pytest.mark.gpu

BYTES = (0, 1, 2, 40, 64, 100, 127, 150, 190, 220, 247, 253, 254)


@pytest.mark.parametrize("code", [0x38, 0x7E, 0x01, 0xB8])
@pytest.mark.parametrize("M", [40, 300])
def test_products_are_exact_at_every_scale(gpu, M, code):
    """One power of two, from the smallest bf16 to the largest, in each row of
    X; one block of each scale byte with one code in all its places.  A result
    is one exact product, rounded once: inf above bf16, also when the scales
    lie far apart."""
    N, K, r = 128 * len(BYTES), 128, 8
    X = torch.zeros(M, K, dtype=torch.float64)
    X[:, 3] = 2.0 ** torch.linspace(-133, 127, M, dtype=torch.float64).round()
    assert torch.equal(X.to(BF16).double(), X)
    Wq = torch.full((N, K), code, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    Ws = torch.tensor(BYTES, dtype=torch.uint8, device="cuda")[:, None].contiguous().view(torch.float8_e8m0fnu)
    A, B = torch.zeros(r, K, dtype=BF16, device="cuda"), torch.zeros(N, r, dtype=BF16, device="cuda")
    Y = torch.full((M, N), float("nan"), dtype=BF16, device="cuda")
    ws = torch.empty(gpu.lora_fp8_workspace_size(M, K, N, r), dtype=torch.uint8, device="cuda")
    gpu.lora_fwd_fp8(X.to(BF16).cuda(), Wq, Ws, A, B, Y, 1.0, ws)
    assert gpu.lora_get_device_status() == 0
    w = Wq[0, 0].float().item() * 2.0 ** (np.array(BYTES, dtype=np.float64) - 127)
    want = torch.tensor(X[:, 3].numpy()[:, None] * w[None]).to(BF16)
    assert torch.equal(Y.cpu().view(M, len(BYTES), 128), want[:, :, None].expand(-1, -1, 128))


def test_a_quantised_layer_after_a_cast_and_a_checkpoint(gpu):
    m = layer(272, 400, 16, 0.0, True, seed=3)
    x = make(50, 272, 400, 16)["X"].cuda()
    want, weight = m(x).detach(), m.base_weight()
    state = {k: v.clone() for k, v in m.state_dict().items()}
    fresh = layer(272, 400, 16, 0.0, False, seed=4)
    fresh.load_state_dict(state)
    for other in (m.to(BF16), m.float().to(BF16), fresh):
        assert torch.equal(other(x), want) and torch.equal(other.base_weight(), weight)
        y = other(x.clone().requires_grad_(True))
        y.sum().backward()
