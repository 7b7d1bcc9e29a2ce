"""lora_fwd_dropout and lora_bwd_dropout against the 64-bit reference: odd
sizes, every rank class, several tiles a cluster, the mask itself, strange
values in dropped places, repeatability and captured replays."""
import numpy as np
import pytest
import torch

import adapter_reference as R

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def make(M, d_in, d_out, r, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = lambda a, b, s: (torch.randn(a, b, generator=g) * s).to(BF16)
    return dict(X=t(M, d_in, 1.0), W=t(d_out, d_in, d_in ** -0.5), A=t(r, d_in, d_in ** -0.5), B=t(d_out, r, 0.1),
                dY=t(M, d_out, 1.0))


def rng_tensor(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def nan_like(shape, dtype=BF16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def run(L, t, scale, p, rng, saved=True, f32=False, backward=True, ws=None):
    d = {k: v.cuda() for k, v in t.items()}
    M, d_in = d["X"].shape
    d_out, r = d["B"].shape
    if ws is None:
        ws = torch.full((max(L.lora_bwd_workspace_size(M, d_in, d_out, r), 256),), 255, dtype=torch.uint8,
                        device="cuda")
    out = {}
    if saved or not backward:
        out["Y"] = nan_like((M, d_out))
        L.lora_fwd_dropout(d["X"], d["W"], d["A"], d["B"], out["Y"], scale, p, rng, ws)
    if backward:
        gdt = torch.float32 if f32 else BF16
        out.update(dX=nan_like((M, d_in)), dA=nan_like((r, d_in), gdt), dB=nan_like((d_out, r), gdt))
        flags = (L.LORA_BWD_T_SAVED if saved else 0) | (L.LORA_BWD_FP32_GRADS if f32 else 0)
        L.lora_bwd_dropout(d["X"], d["W"], d["A"], d["B"], d["dY"], out["dX"], out["dA"], out["dB"], scale, p, rng,
                           ws, flags)
    assert L.lora_get_device_status() == 0
    return out


def host(t):
    return t.double().cpu().numpy()


SIZES = [  # M, d_in, d_out, r, p
    (1, 8, 8, 8, 0.5),
    (3, 136, 72, 8, 0.25),
    (300, 520, 264, 16, 0.1),
    (129, 512, 512, 24, 0.05),
    (257, 1032, 640, 128, 0.3),
    (1000, 264, 1288, 64, 0.9),
    (128, 2048, 256, 40, 0.0),
    (4096, 256, 2048, 32, 0.1),
    (4096, 2048, 256, 32, 0.1),
    # the kernels for few tokens: their limits, long contractions, every split
    (128, 264, 1032, 16, 0.2),
    (17, 4104, 136, 48, 0.3),
    (40, 328, 6408, 128, 0.1),
    (192, 6200, 6216, 8, 0.25),
    (200, 6152, 6152, 32, 0.1),
    (256, 6152, 264, 32, 0.5),
    (512, 136, 264, 16, 0.5),
    (513, 136, 264, 16, 0.5),
]


@pytest.mark.parametrize("M,d_in,d_out,r,p", SIZES)
def test_forward_and_backward_match_the_reference(gpu, M, d_in, d_out, r, p):
    t = make(M, d_in, d_out, r)
    seed, offset = 0x123456789ABCDEF, 77
    rng = rng_tensor(seed, offset) if p > 0 else None
    out = run(gpu, t, 1.5, p, rng)
    mask = R.keep_mask(seed, offset, M, d_in, p) if p > 0 else None
    ref = R.layer(*(R.f64(t[k]) for k in ("X", "W", "A", "B")), 1.5, dY=R.f64(t["dY"]), mask=mask, p=p)
    for name in ("Y", "dB", "dA", "dX"):
        R.check(name, host(out[name]), ref[name])


def test_adapter_alone_shows_the_mask(gpu):
    """W = 0 and A a row of ones at one column: Y is the mask of that column."""
    M, d = 256, 64
    for col in (0, 1, 7, 8, 63):
        X = torch.ones(M, d, dtype=BF16)
        A = torch.zeros(8, d, dtype=BF16)
        A[0, col] = 1
        B = torch.zeros(16, 8, dtype=BF16)
        B[:, 0] = 1
        t = dict(X=X, W=torch.zeros(16, d, dtype=BF16), A=A, B=B, dY=torch.ones(M, 16, dtype=BF16))
        out = run(gpu, t, 1.0, 0.5, rng_tensor(5, 6))
        want = 2.0 * R.keep_mask(5, 6, M, d, 0.5)[:, col].astype(np.float64)
        np.testing.assert_array_equal(host(out["Y"])[:, 3], want)
        # dX's rank product is non-zero in that column alone, under the same mask
        dX = host(out["dX"])
        np.testing.assert_array_equal(dX[:, col], 16 * want)
        assert (np.delete(dX, col, axis=1) == 0).all()


def test_dropped_infinities_and_nan_are_gone(gpu):
    """An infinity or NaN of X in a dropped place reaches nothing but the base
    product; one in a kept place makes T, and so the row, non-finite."""
    M, d, n, r = 64, 128, 64, 8
    t = make(M, d, n, r)
    keep = R.keep_mask(1, 2, M, d, 0.5)
    t["W"].zero_()
    X = t["X"].float().numpy().copy()
    hit = ~keep
    X[hit] = np.where(np.arange(hit.sum()) % 2 == 0, np.inf, np.nan)
    t["X"] = torch.tensor(X).to(BF16)
    t["W"][:, :] = 0
    d_ = {k: v.cuda() for k, v in t.items()}
    ws = torch.empty(gpu.lora_bwd_workspace_size(M, d, n, r), dtype=torch.uint8, device="cuda")
    dX, dA, dB = nan_like((M, d)), nan_like((r, d)), nan_like((n, r))
    gpu.lora_bwd_dropout(d_["X"], d_["W"], d_["A"], d_["B"], d_["dY"], dX, dA, dB, 1.0, 0.5, rng_tensor(1, 2), ws)
    clean = dict(t, X=torch.where(torch.tensor(keep), t["X"], torch.zeros((), dtype=BF16)))
    ref = R.layer(*(R.f64(clean[k]) for k in ("X", "W", "A", "B")), 1.0, dY=R.f64(t["dY"]), mask=keep, p=0.5)
    for name, got in (("dX", dX), ("dA", dA), ("dB", dB)):
        R.check(name, host(got), ref[name])


@pytest.mark.parametrize("f32", [False, True])
def test_recomputed_t_gives_the_saved_results_bit_for_bit(gpu, f32):
    t = make(515, 776, 392, 16)
    a = run(gpu, t, 2.0, 0.2, rng_tensor(9, 1), saved=True, f32=f32)
    b = run(gpu, t, 2.0, 0.2, rng_tensor(9, 1), saved=False, f32=f32)
    for name in ("dX", "dA", "dB"):
        assert torch.equal(a[name], b[name]), name
    if f32:
        c = run(gpu, t, 2.0, 0.2, rng_tensor(9, 1), saved=True)
        for name in ("dA", "dB"):
            assert torch.equal(a[name].to(BF16), c[name]), name


def test_no_dropout_is_the_plain_layer(gpu):
    """p = 0 agrees with lora_fwd_scaled to the roundings of s T."""
    t = make(300, 520, 264, 16)
    out = run(gpu, t, 2.0, 0.0, None, backward=False)
    Y = nan_like((300, 264))
    gpu.lora_fwd_scaled(*(t[k].cuda() for k in ("X", "W", "A", "B")), Y, 2.0)
    assert gpu.lora_get_device_status() == 0
    ref = R.layer(*(R.f64(t[k]) for k in ("X", "W", "A", "B")), 2.0)
    R.check("Y", host(out["Y"]), ref["Y"])
    R.check("Y plain", host(Y), ref["Y"])


def test_empty_batch(gpu):
    t = make(0, 64, 32, 8)
    d = {k: v.cuda() for k, v in t.items()}
    ws = torch.empty(0, dtype=torch.uint8, device="cuda")
    Y, dX, dA, dB = nan_like((0, 32)), nan_like((0, 64)), nan_like((8, 64)), nan_like((32, 8))
    gpu.lora_fwd_dropout(d["X"], d["W"], d["A"], d["B"], Y, 1.0, 0.1, rng_tensor(0, 0), ws)
    gpu.lora_bwd_dropout(d["X"], d["W"], d["A"], d["B"], d["dY"], dX, dA, dB, 1.0, 0.1, rng_tensor(0, 0), ws)
    assert gpu.lora_get_device_status() == 0
    assert (dA == 0).all() and (dB == 0).all()


def test_neighbours_of_the_outputs_stay_as_they_were(gpu):
    M, d_in, d_out, r = 130, 264, 136, 8
    t = make(M, d_in, d_out, r)
    d = {k: v.cuda() for k, v in t.items()}
    need = gpu.lora_bwd_workspace_size(M, d_in, d_out, r)
    guard = 4096
    ws = torch.full((need + guard,), 171, dtype=torch.uint8, device="cuda")
    bufs = {n: torch.full((a * b + 2 * guard,), 7.0, dtype=BF16, device="cuda")
            for n, (a, b) in dict(Y=(M, d_out), dX=(M, d_in), dA=(r, d_in), dB=(d_out, r)).items()}
    view = {n: bufs[n][guard:-guard].view(s) for n, s in dict(Y=(M, d_out), dX=(M, d_in), dA=(r, d_in),
                                                              dB=(d_out, r)).items()}
    rng = rng_tensor(1, 1)
    gpu.lora_fwd_dropout(d["X"], d["W"], d["A"], d["B"], view["Y"], 1.0, 0.1, rng, ws[:need])
    gpu.lora_bwd_dropout(d["X"], d["W"], d["A"], d["B"], d["dY"], view["dX"], view["dA"], view["dB"], 1.0, 0.1, rng,
                         ws[:need], gpu.LORA_BWD_T_SAVED)
    assert gpu.lora_get_device_status() == 0
    assert (ws[need:] == 171).all()
    for n, b in bufs.items():
        assert (b[:guard] == 7).all() and (b[-guard:] == 7).all(), n


def test_captured_step_follows_the_offset(gpu):
    """One captured step, replayed with another offset, draws another mask;
    with the first one it repeats the first results bit for bit."""
    M, d_in, d_out, r, p = 257, 520, 392, 16, 0.25
    t = make(M, d_in, d_out, r)
    d = {k: v.cuda() for k, v in t.items()}
    rng = rng_tensor(3, 0)
    ws = torch.empty(gpu.lora_bwd_workspace_size(M, d_in, d_out, r), dtype=torch.uint8, device="cuda")
    out = dict(Y=nan_like((M, d_out)), dX=nan_like((M, d_in)), dA=nan_like((r, d_in)), dB=nan_like((d_out, r)))

    def step():
        gpu.lora_fwd_dropout(d["X"], d["W"], d["A"], d["B"], out["Y"], 1.0, p, rng, ws)
        gpu.lora_bwd_dropout(d["X"], d["W"], d["A"], d["B"], d["dY"], out["dX"], out["dA"], out["dB"], 1.0, p, rng,
                             ws, gpu.LORA_BWD_T_SAVED)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    first = {k: v.clone() for k, v in out.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    refs = {}
    for offset in (0, 1, 0):
        rng[1] = offset
        graph.replay()
        assert gpu.lora_get_device_status() == 0
        if offset == 0:
            for k, v in out.items():
                assert torch.equal(v, first[k]), k
        else:
            mask = R.keep_mask(3, 1, M, d_in, p)
            refs = R.layer(*(R.f64(t[k]) for k in ("X", "W", "A", "B")), 1.0, dY=R.f64(t["dY"]), mask=mask, p=p)
            for k in out:
                R.check(k, host(out[k]), refs[k])


def test_two_streams_at_once(gpu):
    """Two layers on two streams, each with its own workspace, give what each
    gives alone."""
    ts = [make(700, 1024, 512, 16, seed=s) for s in (1, 2)]
    alone = [run(gpu, t, 1.0, 0.1, rng_tensor(s, s)) for s, t in enumerate(ts)]
    streams = [torch.cuda.Stream() for _ in ts]
    both = [None, None]
    data = [{k: v.cuda() for k, v in t.items()} for t in ts]
    bufs = []
    for s in range(2):
        M, d_in, d_out, r = 700, 1024, 512, 16
        bufs.append((rng_tensor(s, s), torch.empty(gpu.lora_bwd_workspace_size(M, d_in, d_out, r), dtype=torch.uint8,
                                                   device="cuda"),
                     dict(Y=nan_like((M, d_out)), dX=nan_like((M, d_in)), dA=nan_like((r, d_in)),
                          dB=nan_like((d_out, r)))))
    torch.cuda.synchronize()
    for _ in range(4):
        for s in range(2):
            rng, ws, o = bufs[s]
            d = data[s]
            gpu.lora_fwd_dropout(d["X"], d["W"], d["A"], d["B"], o["Y"], 1.0, 0.1, rng, ws, stream=streams[s])
            gpu.lora_bwd_dropout(d["X"], d["W"], d["A"], d["B"], d["dY"], o["dX"], o["dA"], o["dB"], 1.0, 0.1, rng,
                                 ws, gpu.LORA_BWD_T_SAVED, stream=streams[s])
            both[s] = o
    assert gpu.lora_get_device_status() == 0
    for a, b in zip(alone, both):
        for k in a:
            assert torch.equal(a[k], b[k]), k
