"""A row's results do not depend on the batch around it, where two batches
take the same kernels, splits and tiles; and the operators under a compiler
that makes them functional."""
import pytest
import torch

from test_gpu_adapter_dropout import make, rng_tensor, run
from test_gpu_fp8 import quantized, run as run_fp8
from test_gpu_ops_adapter import layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M,first,last", [(1100, 100, 1000), (64, 10, 60)])
def test_rows_of_one_batch_equal_the_same_rows_of_another(gpu, fp8, M, first, last, p):
    """Sizes on one side of every rule: many tokens (pass, tiles) or few (prep,
    stream, 64 token columns).  With a mask, which goes by the row's number,
    the batches begin at the same row."""
    first = 0 if p else first
    t = make(M, 1040, 656, 16)
    part = dict(t, X=t["X"][first:last], dY=t["dY"][first:last])
    rng = rng_tensor(2, 3) if p else None
    if fp8:
        base = quantized(gpu, t["W"])
        a, b = (run_fp8(gpu, u, base, 1.5, p, rng) for u in (t, part))
    else:
        a, b = (run(gpu, u, 1.5, p, rng) for u in (t, part))
    for name in ("Y", "dX"):
        assert torch.equal(a[name][first:last], b[name]), name


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_functionalised_module_equals_eager(gpu, fp8, p):
    """Through torch.compile with functionalisation and a joint graph of
    forward and backward (aot_eager), twice with other inputs."""
    m = layer(512, 256, 16, p, fp8)

    def go(mod, seed):
        t = make(96, 512, 256, 16, seed=seed)
        torch.manual_seed(8)
        m.zero_grad(set_to_none=True)
        x = t["X"].cuda().requires_grad_(True)
        y = mod(x)
        y.backward(t["dY"].cuda())
        return y.detach(), x.grad, m.lora_A.grad, m.lora_B.grad

    torch._dynamo.reset()
    compiled = torch.compile(m, backend="aot_eager", fullgraph=True)
    for seed in (0, 1):
        want = go(m, seed)
        for a, b in zip(want, go(compiled, seed)):
            assert torch.equal(a, b)
