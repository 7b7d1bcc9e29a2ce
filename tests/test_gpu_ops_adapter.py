"""Dropout and the 8-bit base through the torch operators and LoRALinear:
values and gradients against the 64-bit reference and against differences,
stacked layers in a training step, eval mode, repeatability, checkpointing,
capture, torch.compile, strides."""
import numpy as np
import pytest
import torch
from torch.utils.checkpoint import checkpoint

import adapter_reference as R
from test_gpu_adapter_dropout import BF16, host, make, rng_tensor
from test_gpu_fp8 import values

pytestmark = pytest.mark.gpu


def layer(d_in, d_out, r, p, fp8, seed=0):
    from lora_linear_layer_b200 import ops
    g = torch.Generator().manual_seed(seed)
    m = ops.LoRALinear(d_in, d_out, r, 2.0 * r, device="cuda", generator=g, dropout=p)
    with torch.no_grad():
        m.lora_B.copy_((torch.randn(d_out, r, generator=g) * 0.05).to(BF16))
    return m.quantize_base() if fp8 else m


def base_values(m):
    return R.f64(m.weight) if m.weight is not None else values(m.weight_codes, m.weight_scales)


def reference(m, x, dy, rng):
    p = m.dropout if rng is not None else 0.0
    mask = R.keep_mask(int(rng[0]), int(rng[1]), x.shape[0], m.d_in, p) if rng is not None else None
    return R.layer(R.f64(x), base_values(m), R.f64(m.lora_A), R.f64(m.lora_B), m.scale, dY=R.f64(dy), mask=mask, p=p,
                   fp8=m.weight is None)


def draw():
    """What the module draws next from torch's generator of the device."""
    return torch.randint(0, 2 ** 62, (2,), dtype=torch.int64, device="cuda").cpu()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_module_values_and_gradients(gpu, fp8, p):
    m = layer(528, 272, 24, p, fp8)
    x0 = make(3 * 100, 528, 272, 24)["X"].cuda()
    dy = make(3 * 100, 528, 272, 24, seed=5)["dY"].cuda()
    x = x0.reshape(3, 100, 528).clone().requires_grad_(True)
    torch.manual_seed(11)
    rng = draw() if p > 0 else None
    torch.manual_seed(11)
    y = m(x)
    y.backward(dy.reshape(3, 100, 272))
    ref = reference(m, x0, dy, rng)
    for name, got in (("Y", y.reshape(-1, 272)), ("dX", x.grad.reshape(-1, 528)), ("dA", m.lora_A.grad),
                      ("dB", m.lora_B.grad)):
        R.check(name, host(got.detach()), ref[name])


def test_eval_mode_is_the_plain_layer(gpu):
    m = layer(264, 520, 16, 0.5, False).eval()
    x = make(70, 264, 520, 16)["X"].cuda()
    with torch.no_grad():
        want = torch.ops.lora_b200.lora_linear(x, m.weight, m.lora_A, m.lora_B, m.scale)
        assert torch.equal(m(x), want)


def test_quantize_base_keeps_the_weights_values(gpu):
    m = layer(272, 400, 8, 0.0, False)
    w = R.f64(m.weight)
    m.quantize_base()
    assert m.weight is None and "weight_codes" in m.state_dict()
    want = R.quantize(w, 128)[0]
    np.testing.assert_array_equal(base_values(m), want)
    np.testing.assert_array_equal(R.f64(m.base_weight()), want)
    assert m.quantize_base() is m


def test_two_layers_in_a_training_step(gpu):
    """Quantise, then two steps of an up- and a down-projection with dropout:
    every layer's output and gradients against the reference on the inputs
    that it really had."""
    up, down = layer(256, 640, 16, 0.1, True, seed=1), layer(640, 256, 16, 0.1, True, seed=2)
    opt = torch.optim.SGD([q for m in (up, down) for q in m.parameters() if q.requires_grad], lr=1e-3)
    seen = {}
    for step in range(2):
        opt.zero_grad(set_to_none=True)
        x = make(333, 256, 640, 16, seed=step)["X"].cuda().requires_grad_(True)
        torch.manual_seed(100 + step)
        rngs = [draw(), draw()]
        torch.manual_seed(100 + step)
        h = up(x)
        h.retain_grad()
        a = torch.nn.functional.gelu(h)
        a.retain_grad()
        y = down(a)
        dy = make(333, 640, 256, 16, seed=step)["dY"].cuda()
        before = [[q.detach().clone() for q in (m.lora_A, m.lora_B)] for m in (up, down)]
        y.backward(dy)
        for m, xin, out, g_out, g_in, rng in ((down, a, y, dy, a.grad, rngs[1]), (up, x, h, h.grad, x.grad, rngs[0])):
            ref = reference(m, xin.detach(), g_out, rng)
            for name, got in (("Y", out), ("dX", g_in), ("dA", m.lora_A.grad), ("dB", m.lora_B.grad)):
                R.check(name, host(got.detach()), ref[name])
        opt.step()
        seen[step] = before
    assert not torch.equal(seen[0][0][0], seen[1][0][0])


@pytest.mark.parametrize("fp8", [False, True])
def test_gradients_against_differences(gpu, fp8):
    """The layer is linear in A, and in B: <dY, Y(A + D) - Y(A - D)> / 2 is
    <dA, D>, up to the bounds of the four results.  Over a bf16 base it is
    linear in X too."""
    M, K, N, r, s, p = 200, 512, 384, 16, 1.0, 0.3
    t = make(M, K, N, r)
    from lora_linear_layer_b200 import ops
    d = {k: v.cuda() for k, v in t.items()}
    W, Ws = ops.quantize_weight(d["W"]) if fp8 else (d["W"], None)
    Wv = values(W, Ws) if fp8 else R.f64(W)
    rng = rng_tensor(4, 4)
    mask = R.keep_mask(4, 4, M, K, p)

    def forward(X, A, B):
        Y = torch.ops.lora_b200.lora_linear_adapter(X, W, Ws, A, B, s, p, rng)[0]
        bound = R.layer(R.f64(X), Wv, R.f64(A), R.f64(B), s, mask=mask, p=p, fp8=fp8)["Y"][1]
        return host(Y), bound

    Y, saved = torch.ops.lora_b200.lora_linear_adapter(d["X"], W, Ws, d["A"], d["B"], s, p, rng)
    grads = dict(zip("XAB", torch.ops.lora_b200.lora_linear_adapter_bwd(d["X"], W, Ws, d["A"], d["B"], d["dY"], saved,
                                                                        s, p, rng, True)))
    bounds = R.layer(R.f64(t["X"]), Wv, R.f64(t["A"]), R.f64(t["B"]), s, dY=R.f64(t["dY"]), mask=mask, p=p, fp8=fp8)
    dY = R.f64(t["dY"])
    g = torch.Generator().manual_seed(1)
    for name in ("A", "B") if fp8 else ("A", "B", "X"):
        here = t[name].float()
        # (the two points are rounded to bf16; being linear, the difference asks
        # only for the step between them)
        D = torch.randint(-3, 4, here.shape, generator=g) * torch.exp2(torch.floor(torch.log2(here.abs().clamp_min(
            1e-6))) - 4)
        hi, lo = (here + D).to(BF16), (here - D).to(BF16)
        step = (R.f64(hi) - R.f64(lo)) / 2
        (yh, bh), (yl, bl) = (forward(*(v.cuda() if n == name else d[n] for n in "XAB")) for v in (hi, lo))
        got = (dY * (yh - yl)).sum() / 2
        want = (host(grads[name]) * step).sum()
        slack = (np.abs(dY) * (bh + bl)).sum() / 2 + (bounds["d" + name][1] * np.abs(step)).sum()
        assert abs(got - want) <= slack, (name, got, want, slack)


def test_same_seed_same_run_and_checkpointing(gpu):
    m = layer(256, 384, 16, 0.3, True)
    x0 = make(150, 256, 384, 16)["X"].cuda()
    dy = make(150, 256, 384, 16)["dY"].cuda()

    def go(call):
        torch.manual_seed(3)
        m.zero_grad(set_to_none=True)
        x = x0.clone().requires_grad_(True)
        y = call(x)
        torch.rand(5, device="cuda")  # something else draws in between
        y.backward(dy)
        return y.detach(), x.grad, m.lora_A.grad, m.lora_B.grad

    first = go(m)
    for other in (go(m), go(lambda x: checkpoint(m, x, use_reentrant=False))):
        for a, b in zip(first, other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_training_step_draws_new_masks(gpu, fp8):
    m = layer(256, 384, 16, 0.5, fp8)
    x = make(130, 256, 384, 16)["X"].cuda().requires_grad_(True)
    dy = make(130, 256, 384, 16)["dY"].cuda()
    args = (m.weight if m.weight is not None else m.weight_codes, None if m.weight is not None else m.weight_scales)

    def step():
        rng = torch.randint(0, 2 ** 62, (2,), dtype=torch.int64, device="cuda")
        y, _ = torch.ops.lora_b200.lora_linear_adapter(x, *args, m.lora_A, m.lora_B, m.scale, 0.5, rng)
        grads = torch.autograd.grad(y, (x, m.lora_A, m.lora_B), dy)
        return (rng, y.detach(), *grads)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # no eager graph of these leaves is alive at capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    masks = []
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        rng = out[0].cpu()
        ref = reference(m, x.detach(), dy, rng)
        for name, got in zip(("Y", "dX", "dA", "dB"), out[1:]):
            R.check(name, host(got), ref[name])
        masks.append(tuple(rng.tolist()))
    assert masks[0] != masks[1]


@pytest.mark.parametrize("fp8", [False, True])
def test_compiled_fullgraph_equals_eager(gpu, fp8):
    m = layer(512, 256, 16, 0.1, fp8)
    x0 = make(96, 512, 256, 16)["X"].cuda()
    dy = make(96, 512, 256, 16)["dY"].cuda()

    def go(mod):
        torch.manual_seed(8)
        m.zero_grad(set_to_none=True)
        x = x0.clone().requires_grad_(True)
        y = mod(x)
        y.backward(dy)
        return y.detach(), x.grad, m.lora_A.grad, m.lora_B.grad

    eager = go(m)
    torch._dynamo.reset()
    for a, b in zip(eager, go(torch.compile(m, backend="eager", fullgraph=True))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fp8", [False, True])
def test_opcheck(gpu, fp8):
    from lora_linear_layer_b200 import ops
    t = {k: v.cuda() for k, v in make(40, 64, 48, 8).items()}
    W, Ws = ops.quantize_weight(t["W"]) if fp8 else (t["W"], None)
    X, A, B = (t[k].requires_grad_(True) for k in ("X", "A", "B"))
    torch.library.opcheck(torch.ops.lora_b200.lora_linear_adapter.default, (X, W, Ws, A, B, 1.0, 0.1, rng_tensor(1, 2)),
                          # (the schema test does arithmetic on its inputs, which torch lacks for e4m3)
                          test_utils=(() if fp8 else ("test_schema",)) + ("test_faketensor", "test_autograd_registration"))


def test_strided_and_shared_inputs(gpu):
    """A transposed input, a gradient that is a broadcast, and one adapter
    used twice in a graph (its gradients add up)."""
    m = layer(256, 256, 8, 0.25, True)
    x = make(96, 256, 256, 8)["X"].cuda()
    xt = x.t().contiguous().t()
    assert not xt.is_contiguous()
    torch.manual_seed(1)
    a = m(x)
    torch.manual_seed(1)
    assert torch.equal(a, m(xt))
    torch.manual_seed(2)
    rngs = [draw(), draw()]
    torch.manual_seed(2)
    y1 = m(x)
    y2 = m(y1.detach())
    (y1.sum() + y2.sum()).backward()  # the gradients of a sum are an expanded one
    ones = torch.ones(96, 256, dtype=BF16)
    r1, r2 = reference(m, x, ones, rngs[0]), reference(m, y1.detach(), ones, rngs[1])
    for name, got in (("dA", m.lora_A.grad), ("dB", m.lora_B.grad)):
        v = r1[name][0] + r2[name][0]
        bound = r1[name][1] + r2[name][1] + R.HALF_BF16 * (np.abs(v) + r1[name][1] + r2[name][1])
        R.check(name, host(got), (v, bound))


def test_tensors_of_a_call_share_a_device(gpu):
    t = {k: v.cuda() for k, v in make(8, 64, 64, 8).items()}
    Y = torch.empty(8, 64, dtype=BF16, device="cuda")
    ws = torch.empty(gpu.lora_bwd_workspace_size(8, 64, 64, 8), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        gpu.lora_fwd_dropout(t["X"], t["W"], t["A"].cpu(), t["B"], Y, 1.0, 0.1, rng_tensor(0, 0), ws)
    with pytest.raises(ValueError):
        gpu.lora_fwd_dropout(t["X"], t["W"], t["A"], t["B"], Y, 1.0, 0.1, rng_tensor(0, 0).cpu(), ws)
    with pytest.raises(ValueError):
        gpu.lora_fwd_dropout(t["X"], t["W"], t["A"], t["B"], Y.t(), 1.0, 0.1, rng_tensor(0, 0), ws)
    with pytest.raises(gpu.LoraError):
        gpu.lora_fwd_dropout(t["X"], t["W"], t["A"], t["B"], Y, 1.0, 0.1, rng_tensor(0, 0), ws[:256])


def test_missing_tensors_are_named(gpu):
    t = {k: v.cuda() for k, v in make(8, 64, 64, 8).items()}
    Y = torch.empty(8, 64, dtype=BF16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    codes = t["W"].to(torch.float8_e4m3fn)
    for missing in (None, 3):
        with pytest.raises(TypeError, match="Ws"):
            gpu.lora_fwd_fp8(t["X"], codes, missing, t["A"], t["B"], Y, 1.0, ws)
        with pytest.raises(TypeError, match="Wq"):
            gpu.lora_quantize_fp8(t["W"], missing, missing)
        with pytest.raises(TypeError, match="workspace"):
            gpu.lora_fwd_dropout(t["X"], t["W"], t["A"], t["B"], Y, 1.0, 0.1, rng_tensor(0, 0), missing)
        with pytest.raises(TypeError, match="A must"):
            gpu.lora_fwd_dropout(t["X"], t["W"], missing, t["B"], Y, 1.0, 0.1, rng_tensor(0, 0), ws)
    with pytest.raises(gpu.LoraError):
        gpu.lora_fwd_dropout(t["X"], t["W"], t["A"], t["B"], Y, 1.0, 0.1, None, ws)


def test_scale_and_p_may_be_any_number(gpu):
    t = {k: v.cuda() for k, v in make(8, 64, 64, 8).items()}
    ws = torch.empty(gpu.lora_bwd_workspace_size(8, 64, 64, 8), dtype=torch.uint8, device="cuda")
    out = []
    for scale, p in ((2.0, 0.25), (2, np.float32(0.25)), (np.float32(2.0), torch.tensor(0.25)), (torch.tensor(2.0), 0.25)):
        Y = torch.empty(8, 64, dtype=BF16, device="cuda")
        gpu.lora_fwd_dropout(t["X"], t["W"], t["A"], t["B"], Y, scale, p, rng_tensor(3, 4), ws)
        out.append(Y)
    assert all(torch.equal(Y, out[0]) for Y in out)


@pytest.mark.parametrize("M", [1, 200])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_forward_that_saves_nothing(gpu, fp8, M):
    """The same Y, no T; and a backward all the same, from T computed again."""
    from lora_linear_layer_b200 import ops

    t = {k: v.cuda() for k, v in make(M, 272, 400, 16).items()}
    W, Ws = ops.quantize_weight(t["W"]) if fp8 else (t["W"], None)
    rng = rng_tensor(5, 6)
    results = []
    for save in (True, False):
        X, A, B = (t[k].clone().requires_grad_(True) for k in "XAB")
        Y, saved = torch.ops.lora_b200.lora_linear_adapter(X, W, Ws, A, B, 2.0, 0.25, rng, save)
        assert (saved.numel() > 0) == save
        results.append((Y, *torch.autograd.grad(Y, (X, A, B), t["dY"])))
    for got, want in zip(*results):
        assert torch.equal(got, want)


@pytest.mark.parametrize("fp8", [False, True])
def test_module_saves_only_for_a_backward(gpu, fp8):
    m = layer(272, 400, 16, 0.0, fp8)
    x = make(3, 272, 400, 16)["X"].cuda()
    y = m(x)
    with torch.no_grad():
        assert torch.equal(m(x), y.detach())
    assert y.requires_grad


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M", [5, 200, 1300])
def test_queued_steps_that_feed_each_other(gpu, fp8, M):
    """Steps queued one behind another on one workspace, each with a weight
    that was written just before it and the dX of the step before as its dY:
    the results of the same steps with a wait after every call, bit for bit."""
    L, d, r, steps = gpu, 768, 16, 12
    g = torch.Generator().manual_seed(3)
    rand = lambda *shape: (torch.randn(*shape, generator=g) * shape[-1] ** -0.5).to(BF16).cuda()
    weights, inputs = [rand(d, d) for _ in range(steps)], [rand(M, d) * 20 for _ in range(steps)]
    A, B, first = rand(r, d), rand(d, r), rand(M, d) * 20
    size = (L.lora_fp8_workspace_size if fp8 else L.lora_bwd_workspace_size)(M, d, d, r)
    rng = rng_tensor(11, 12)

    def run(wait):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        W = torch.zeros(d, d, dtype=BF16, device="cuda")
        Wq = torch.zeros(d, d, dtype=torch.float8_e4m3fn, device="cuda")
        Ws = torch.zeros(d // 128, d // 128, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
        out = [{n: torch.empty(*shape, dtype=BF16, device="cuda")
                for n, shape in (("Y", (M, d)), ("dX", (M, d)), ("dA", (r, d)), ("dB", (d, r)))} for _ in range(steps)]
        dY = first
        torch.cuda.synchronize()
        for X, new, o in zip(inputs, weights, out):
            calls = []
            if fp8:
                calls.append(lambda: L.lora_quantize_fp8(new, Wq, Ws))
                calls.append(lambda: L.lora_fwd_fp8(X, Wq, Ws, A, B, o["Y"], 2.0, ws, 0.25, rng))
                calls.append(lambda: L.lora_bwd_fp8(X, Wq, Ws, A, B, dY, o["dX"], o["dA"], o["dB"], 2.0, ws, 0.25, rng,
                                                    L.LORA_BWD_T_SAVED))
            else:
                calls.append(lambda: L.lora_restore(new, W))
                calls.append(lambda: L.lora_fwd_dropout(X, W, A, B, o["Y"], 2.0, 0.25, rng, ws))
                calls.append(lambda: L.lora_bwd_dropout(X, W, A, B, dY, o["dX"], o["dA"], o["dB"], 2.0, 0.25, rng, ws,
                                                        L.LORA_BWD_T_SAVED))
            for call in calls:
                call()
                if wait:
                    torch.cuda.synchronize()
            dY = o["dX"]
        torch.cuda.synchronize()
        return out

    want = run(True)
    assert all(torch.isfinite(t.float()).all() for o in want for t in o.values())
    for _ in range(10):
        for o, w in zip(run(False), want):
            for n in w:
                assert torch.equal(o[n], w[n]), n
    assert L.lora_get_device_status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_module_on_an_empty_batch(gpu, fp8):
    m = layer(64, 48, 8, 0.1, fp8)
    x = torch.empty(2, 0, 64, dtype=BF16, device="cuda", requires_grad=True)
    y = m(x)
    assert y.shape == (2, 0, 48)
    y.sum().backward()
    assert x.grad.shape == x.shape and (m.lora_A.grad == 0).all() and (m.lora_B.grad == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_backward_twice_through_one_graph(gpu, fp8):
    m = layer(256, 136 if not fp8 else 144, 8, 0.2, fp8)
    x = make(77, 256, m.d_out, 8)["X"].cuda().requires_grad_(True)
    y = m(x)
    dy = torch.ones_like(y)
    first = torch.autograd.grad(y, (x, m.lora_A, m.lora_B), dy, retain_graph=True)
    for a, b in zip(first, torch.autograd.grad(y, (x, m.lora_A, m.lora_B), dy)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(gpu, fp8):
    """X of 2.4 * 10^9 elements: rows on both sides of 2^31 elements, and the
    last, against the reference."""
    from lora_linear_layer_b200 import ops
    M, K, N, r, p = 590001, 4096, 64, 8, 0.25
    t = make(8, K, N, r)
    g = torch.Generator(device="cuda").manual_seed(0)
    X = torch.empty(M, K, dtype=BF16, device="cuda")
    for i in range(0, M, 65536):
        X[i:i + 65536] = torch.randn(min(65536, M - i), K, generator=g, device="cuda").to(BF16)
    W, A, B = (t[k].cuda() for k in ("W", "A", "B"))
    Wq, Ws = ops.quantize_weight(W) if fp8 else (W, None)
    rng = rng_tensor(7, 8)
    Y, saved = torch.ops.lora_b200.lora_linear_adapter(X, Wq, Ws, A, B, 1.0, p, rng)
    dY = torch.ones(M, N, dtype=BF16, device="cuda")
    dX, _, _ = torch.ops.lora_b200.lora_linear_adapter_bwd(X, Wq, Ws, A, B, dY, saved, 1.0, p, rng)
    assert gpu.lora_get_device_status() == 0
    edge = 2 ** 31 // K
    rows = torch.tensor([0, 127, edge - 1, edge, edge + 1, M - 130, M - 1])
    keep = np.concatenate([R.keep_mask(7, 8, 1, K, p) if i == 0 else _mask_row(7, 8, int(i), K, p) for i in rows])
    Wv = values(Wq, Ws) if fp8 else R.f64(W)
    ref = R.layer(R.f64(X[rows.cuda()]), Wv, R.f64(A), R.f64(B), 1.0, dY=np.ones((len(rows), N)), mask=keep, p=p,
                  fp8=fp8)
    R.check("Y", host(Y[rows.cuda()]), ref["Y"])
    R.check("dX", host(dX[rows.cuda()]), ref["dX"])


def _mask_row(seed, offset, i, K, p):
    words = R.philox(np.arange(K // 8), np.full(K // 8, i), np.full(K // 8, offset), np.zeros(K // 8, dtype=int), seed, 0)
    lanes = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], axis=-1)
    return (lanes.reshape(1, K) >= R.threshold(p))
