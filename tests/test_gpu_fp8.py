"""The 8-bit base: its conversion, and the layer over it, against the 64-bit
reference."""
import numpy as np
import pytest
import torch

import adapter_reference as R
from test_gpu_adapter_dropout import BF16, host, make, nan_like, rng_tensor

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu


def codes_like(d_out, d_in):
    nb, kb = (d_out + 127) // 128, (d_in + 127) // 128
    return (torch.full((d_out, d_in), 77, dtype=torch.uint8, device="cuda").view(E4M3),
            torch.full((nb, kb), 77, dtype=torch.uint8, device="cuda").view(E8M0))


def quantized(L, W):
    Wq, Ws = codes_like(*W.shape)
    L.lora_quantize_fp8(W.cuda(), Wq, Ws)
    return Wq, Ws


def values(Wq, Ws):
    """fp64 values of codes and scales, on the host."""
    s = 2.0 ** (Ws.view(torch.uint8).cpu().double().numpy() - 127)
    n, k = Wq.shape
    return Wq.float().cpu().double().numpy() * np.kron(s, np.ones((128, 128)))[:n, :k]


@pytest.mark.parametrize("d_out,d_in", [(1, 16), (128, 128), (130, 144), (129, 1040), (640, 272), (2000, 512)])
def test_weight_conversion(gpu, d_out, d_in):
    g = torch.Generator().manual_seed(d_out)
    W = (torch.randn(d_out, d_in, generator=g) * torch.exp2(torch.randint(-30, 30, (d_out, 1), generator=g).float())
         ).to(BF16)
    Wq, Ws = quantized(gpu, W)
    assert gpu.lora_get_device_status() == 0
    want, e = R.quantize(R.f64(W), 128)
    np.testing.assert_array_equal(Ws.view(torch.uint8).cpu().numpy().astype(int) - 127, e)
    np.testing.assert_array_equal(values(Wq, Ws), want)
    back = nan_like((d_out, d_in))
    gpu.lora_dequantize_fp8(Wq, Ws, back)
    assert torch.equal(back.cpu(), torch.tensor(want, dtype=torch.float64).to(BF16))


def test_weight_conversion_at_the_edges_of_the_range(gpu):
    """Zero blocks, the largest and the smallest magnitudes, values on a
    boundary between two scales, infinities and NaN."""
    W = torch.zeros(128 * 8, 128, dtype=BF16)
    tops = [0.0, 448.0, 450.0, 446.0, torch.finfo(BF16).max, 2.0 ** -133, 1.75 * 2.0 ** -120]
    for i, v in enumerate(tops):
        W[128 * i, 5] = v
        W[128 * i + 127, 127] = -v / 2
    W[128 * 7 + 3, 9] = float("inf")
    Wq, Ws = quantized(gpu, W)
    e = R.exponents(np.array([abs(float(torch.tensor(v).to(BF16))) for v in tops]))
    b = Ws.view(torch.uint8).cpu().numpy()[:, 0]
    np.testing.assert_array_equal(b[:7].astype(int) - 127, e)
    assert b[7] == 255
    want = R.quantize(R.f64(W[:896]), 128)[0]
    np.testing.assert_array_equal(values(Wq[:896], Ws[:7]), want)
    back = nan_like(tuple(W.shape))
    gpu.lora_dequantize_fp8(Wq, Ws, back)
    assert torch.equal(back[:896].cpu(), torch.tensor(want).to(BF16)) and back[896:].isnan().all()
    W[128 * 7 + 3, 9] = float("nan")
    assert quantized(gpu, W)[1].view(torch.uint8)[7, 0] == 255


def run(L, t, base, scale, p=0.0, rng=None, backward=True, saved=True, f32=False):
    d = {k: v.cuda() for k, v in t.items()}
    Wq, Ws = base
    M, d_in = d["X"].shape
    d_out, r = d["B"].shape
    ws = torch.full((L.lora_fp8_workspace_size(M, d_in, d_out, r),), 255, dtype=torch.uint8, device="cuda")
    out = {}
    if saved or not backward:
        out["Y"] = nan_like((M, d_out))
        L.lora_fwd_fp8(d["X"], Wq, Ws, d["A"], d["B"], out["Y"], scale, ws, p, rng)
    if backward:
        gdt = torch.float32 if f32 else BF16
        out.update(dX=nan_like((M, d_in)), dA=nan_like((r, d_in), gdt), dB=nan_like((d_out, r), gdt))
        flags = (L.LORA_BWD_T_SAVED if saved else 0) | (L.LORA_BWD_FP32_GRADS if f32 else 0)
        L.lora_bwd_fp8(d["X"], Wq, Ws, d["A"], d["B"], d["dY"], out["dX"], out["dA"], out["dB"], scale, ws, p, rng,
                       flags)
    assert L.lora_get_device_status() == 0
    return out


SIZES = [  # M, d_in, d_out, r, p
    (1, 16, 16, 8, 0.0),
    (1, 512, 256, 16, 0.0),
    (5, 1040, 272, 24, 0.5),
    (16, 2048, 304, 16, 0.0),
    (33, 640, 1040, 128, 0.0),
    (300, 528, 272, 16, 0.1),
    (129, 512, 512, 24, 0.0),
    (257, 1040, 640, 128, 0.3),
    (1000, 272, 1296, 64, 0.0),
    (4096, 256, 2048, 32, 0.1),
    (4096, 2048, 256, 32, 0.0),
    # the kernels for few tokens: their limits, long contractions, every split
    (128, 272, 1040, 16, 0.2),
    (17, 4112, 144, 48, 0.3),
    (40, 336, 6416, 128, 0.0),
    (192, 6192, 6208, 8, 0.25),
    (200, 6160, 6160, 32, 0.1),
    (256, 6160, 272, 32, 0.0),
    (64, 128, 128, 128, 0.5),
    (65, 128, 128, 128, 0.5),
]


@pytest.mark.parametrize("M,d_in,d_out,r,p", SIZES)
def test_forward_and_backward_match_the_reference(gpu, M, d_in, d_out, r, p):
    t = make(M, d_in, d_out, r)
    # rows and columns of very unequal strength: every group has its own scale
    g = torch.Generator().manual_seed(1)
    t["X"] = (t["X"].float() * torch.exp2(torch.randint(-6, 7, (M, 1), generator=g).float())
              * torch.exp2(torch.randint(-4, 5, (1, d_in), generator=g).float())).to(BF16)
    t["W"] = (t["W"].float() * torch.exp2(torch.arange(d_out)[:, None] // 128 % 5 - torch.arange(d_in)[None] // 128 % 7
                                          ).float()).to(BF16)
    base = quantized(gpu, t["W"])
    seed, offset = -5, 1 << 40
    out = run(gpu, t, base, 1.5, p, rng_tensor(seed, offset) if p > 0 else None)
    mask = R.keep_mask(seed, offset, M, d_in, p) if p > 0 else None
    W = values(*base)
    ref = R.layer(R.f64(t["X"]), W, R.f64(t["A"]), R.f64(t["B"]), 1.5, dY=R.f64(t["dY"]), mask=mask, p=p, fp8=True)
    for name in ("Y", "dB", "dA", "dX"):
        R.check(name, host(out[name]), ref[name])


@pytest.mark.parametrize("M", [1, 7, 40, 300])
def test_one_strong_value_in_each_scale_group(gpu, M):
    """B = 0 and one non-zero value of X in each group: Y is W's values times
    powers of two, so a scale taken from another row, column or group shows
    as a wrong power."""
    d_in, d_out, r = 1040, 528, 8
    t = make(M, d_in, d_out, r)
    t["B"].zero_()
    g = torch.Generator().manual_seed(2)
    for group in range(9):
        X = torch.zeros(M, d_in, dtype=BF16)
        cols = torch.randint(128 * group, min(128 * (group + 1), d_in), (M,), generator=g)
        powers = torch.randint(-40, 40, (M,), generator=g)
        X[torch.arange(M), cols] = torch.exp2(powers.float()).to(BF16)
        t["W"] = torch.exp2(torch.randint(-3, 4, (d_out, d_in), generator=g).float()
                            + (torch.arange(d_out)[:, None] // 128 * 11 - torch.arange(d_in)[None] // 128 * 7)).to(BF16)
        t["X"] = X
        base = quantized(gpu, t["W"])
        out = run(gpu, t, base, 1.0, backward=False)
        want = R.f64(X) @ values(*base).T
        np.testing.assert_array_equal(host(out["Y"]), want)


@pytest.mark.parametrize("M", [1, 200])
def test_non_finite_rows_stay_in_their_rows(gpu, M):
    d_in, d_out, r = 512, 256, 16
    t = make(M + 1, d_in, d_out, r)
    base = quantized(gpu, t["W"])
    clean = run(gpu, t, base, 1.0, backward=False)["Y"]
    t["X"][M, 300] = float("inf")
    t["X"][0, 5] = float("nan")
    Y = run(gpu, t, base, 1.0, backward=False)["Y"]
    assert Y[0].isnan().all() and Y[M].isnan().all()
    assert torch.equal(Y[1:M], clean[1:M])


@pytest.mark.parametrize("p", [0.0, 0.2])
def test_recomputed_t_gives_the_saved_results_bit_for_bit(gpu, p):
    t = make(515, 784, 400, 16)
    base = quantized(gpu, t["W"])
    rng = rng_tensor(9, 1) if p else None
    a = run(gpu, t, base, 2.0, p, rng, saved=True, f32=True)
    b = run(gpu, t, base, 2.0, p, rng, saved=False, f32=True)
    for name in ("dX", "dA", "dB"):
        assert torch.equal(a[name], b[name]), name
    c = run(gpu, t, base, 2.0, p, rng)
    for name in ("dA", "dB"):
        assert torch.equal(a[name].to(BF16), c[name]), name


def test_empty_batch(gpu):
    t = make(0, 64, 32, 8)
    base = quantized(gpu, t["W"])
    d = {k: v.cuda() for k, v in t.items()}
    ws = torch.empty(0, dtype=torch.uint8, device="cuda")
    gpu.lora_fwd_fp8(d["X"], *base, d["A"], d["B"], nan_like((0, 32)), 1.0, ws)
    dA, dB = nan_like((8, 64)), nan_like((32, 8))
    gpu.lora_bwd_fp8(d["X"], *base, d["A"], d["B"], d["dY"], nan_like((0, 64)), dA, dB, 1.0, ws)
    assert gpu.lora_get_device_status() == 0
    assert (dA == 0).all() and (dB == 0).all()


def test_a_row_does_not_depend_on_its_batch(gpu):
    """Rows of one call of a kernel equal the same rows of another batch."""
    t = make(600, 1040, 656, 16)
    base = quantized(gpu, t["W"])
    whole = run(gpu, t, base, 1.0, backward=False)["Y"]
    part = run(gpu, dict(t, X=t["X"][100:500], dY=t["dY"][100:500]), base, 1.0, backward=False)["Y"]
    ref = R.layer(R.f64(t["X"]), values(*base), R.f64(t["A"]), R.f64(t["B"]), 1.0, fp8=True)["Y"]
    R.check("whole", host(whole), ref)
    R.check("part", host(part), (ref[0][100:500], ref[1][100:500]))


def test_captured_token_step(gpu):
    """A captured single-token forward reads the inputs of each replay."""
    M, d_in, d_out, r = 1, 1024, 768, 16
    t = make(M, d_in, d_out, r)
    base = quantized(gpu, t["W"])
    d = {k: v.cuda() for k, v in t.items()}
    ws = torch.empty(gpu.lora_fp8_workspace_size(M, d_in, d_out, r), dtype=torch.uint8, device="cuda")
    Y = nan_like((M, d_out))
    call = lambda: gpu.lora_fwd_fp8(d["X"], *base, d["A"], d["B"], Y, 1.0, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(3):
        X = make(M, d_in, d_out, r, seed=seed)["X"]
        d["X"].copy_(X)
        graph.replay()
        assert gpu.lora_get_device_status() == 0
        ref = R.layer(R.f64(X), values(*base), R.f64(t["A"]), R.f64(t["B"]), 1.0, fp8=True)
        R.check("Y", host(Y), ref["Y"])
