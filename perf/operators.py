"""Cases and plain forms of the adapter-dropout and 8-bit-base operators.

    dropout   Y  = X W^T + s/(1-p) ((m * X) A^T) B^T           (bf16 base)
    fp8       Y  = Xq Wq^T + s/(1-p) ((m * X) A^T) B^T         (8-bit base)
    backward  dT = s dY B,  dB = dY^T T,  dA = dT^T (m * X)/(1-p),
              dX = dY W (or dYq Wq) + m * (dT A)/(1-p),  T = s/(1-p) (m * X) A^T
    quantize  W -> e4m3 codes with one power-of-two scale for each 128 x 128 block, and back

m is the dropout mask.  It is never stored: element (i, k) is kept when the
16-bit lane k % 8 of the Philox4x32-7 block with counter (k / 8, i, offset)
and key seed is at least round(65536 p), and p then stands for that
threshold over 65536.  Xq and dYq hold X and dY rounded to e4m3 with one
power-of-two scale for each row and each 128 values of the contraction: the
smallest scale with which the group's largest magnitude is at most 448.

Work counts each input and output once and every product at 2 operations a
multiply-add.  All sizes are those of the repository's own workloads, or odd
ones of the same range.
"""
import functools
import math

import numpy as np
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0


# ----------------------------------------------------------------- cases ----

def listed():
    return [
        # the tiny forward of the benchmark, with the adapter's usual dropout: launch latency counts
        dict(name="dropout_fwd_tiny", op="dropout_fwd", M=256, d_in=512, d_out=512, r=16, p=0.05, scale=2.0),
        # the attention projection, batch 4 x 2048 tokens
        dict(name="dropout_fwd_attn", op="dropout_fwd", M=8192, d_in=4096, d_out=4096, r=16, p=0.1, scale=2.0),
        # a ragged packed batch through an MLP projection of the merge workload, forward and backward
        dict(name="dropout_train_ragged", op="dropout_train", M=1237, d_in=2560, d_out=9728, r=24, p=0.05, scale=5.656854),
        # the MLP up-projection training step
        dict(name="dropout_train_mlp", op="dropout_train", M=16384, d_in=4096, d_out=14336, r=64, p=0.1, scale=2.0),
        # one generated token through an attention projection with an active adapter
        dict(name="fp8_fwd_token", op="fp8_fwd", M=1, d_in=4096, d_out=4096, r=16, p=0.0, scale=2.0),
        # a decode batch of an odd size through an MLP projection
        dict(name="fp8_fwd_decode", op="fp8_fwd", M=23, d_in=2560, d_out=9728, r=32, p=0.0, scale=2.0),
        # a prompt through a wide square layer
        dict(name="fp8_fwd_prompt", op="fp8_fwd", M=512, d_in=8192, d_out=8192, r=16, p=0.0, scale=2.0),
        # the attention projection over the 8-bit base
        dict(name="fp8_fwd_attn", op="fp8_fwd", M=8192, d_in=4096, d_out=4096, r=16, p=0.0, scale=2.0),
        # a ragged batch, a narrow key/value projection, the largest rank, forward and backward
        dict(name="fp8_train_kv", op="fp8_train", M=2051, d_in=2560, d_out=1024, r=128, p=0.0, scale=1.0),
        # the MLP up-projection training step over the 8-bit base, with dropout
        dict(name="fp8_train_mlp", op="fp8_train", M=16384, d_in=4096, d_out=14336, r=64, p=0.05, scale=2.0),
        # a key/value projection's weight to 8 bits and back
        dict(name="quantize_kv", op="quantize", d_in=2560, d_out=1024),
        # the MLP up-projection's weight to 8 bits and back
        dict(name="quantize_mlp", op="quantize", d_in=4096, d_out=14336),
    ]


def draw(rng):
    op = rng.choice(["dropout_fwd", "dropout_train", "fp8_fwd", "fp8_fwd", "fp8_train", "quantize"])
    step = 8 if op.startswith("dropout") else 16
    spread = lambda lo, hi: math.exp(rng.uniform(math.log(lo), math.log(hi)))
    d_in = max(step, int(spread(256, 14336)) // step * step)
    d_out = max(step, int(spread(256, 14336)) // step * step)
    if op == "quantize":
        return dict(op=op, d_in=d_in, d_out=d_out)
    most = 16384 * 4096 * 14336 // (d_in * d_out)
    least = 16 if op.endswith("train") else 1
    M = int(spread(least, min(16384, most)))
    p = rng.choice([0.0, 0.05, 0.1, 0.3]) if op.startswith("fp8") else rng.choice([0.01, 0.05, 0.1, 0.3, 0.5])
    return dict(op=op, M=M, d_in=d_in, d_out=d_out, r=8 * rng.randint(1, 16), p=p, scale=rng.choice([0.5, 1.0, 2.0, 4.0]))


def work(case):
    k, n = case["d_in"], case["d_out"]
    blocks = -(-k // BLOCK) * -(-n // BLOCK)
    if case["op"] == "quantize":
        return {"bytes": 5 * k * n + blocks, "flops": 2 * k * n}
    m, r = case["M"], case["r"]
    base = k * n * (1 if case["op"].startswith("fp8") else 2) + (blocks if case["op"].startswith("fp8") else 0)
    data = base + 2 * (m * k + r * k + n * r + m * n)
    flops = 2 * m * k * n + 2 * m * r * (k + n)
    if case["op"].endswith("train"):
        data += 2 * (m * n + m * k + r * k + n * r)
        flops += 2 * m * k * n + 4 * m * r * (k + n)
    return {"bytes": data, "flops": flops}


# ---------------------------------------------------------------- inputs ----

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    k, n = case["d_in"], case["d_out"]
    normal = lambda rows, cols, std: (torch.randn(rows, cols, generator=g, device=dev) * std).bfloat16()
    state = {"case": dict(case)}
    W = normal(n, k, k ** -0.5)
    if case["op"] == "quantize":
        state["W"] = W
        state["Wq"] = torch.empty(n, k, dtype=torch.float8_e4m3fn, device=dev)
        state["Ws"] = torch.empty(-(-n // BLOCK), -(-k // BLOCK), dtype=torch.float8_e8m0fnu, device=dev)
        state["out"] = torch.empty_like(W)
        return state
    m, r = case["M"], case["r"]
    # channels of unequal strength, as the inputs of a trained layer have them
    channel = torch.exp(0.5 * torch.randn(1, k, generator=g, device=dev))
    state["X"] = (torch.randn(m, k, generator=g, device=dev) * channel).bfloat16()
    state["A"], state["B"] = normal(r, k, k ** -0.5), normal(n, r, 0.02)
    if case["op"].startswith("fp8"):
        state["Wq"], state["Ws"] = _quantize(W)
    else:
        state["W"] = W
    state["rng"] = torch.tensor([(seed * 7919 + 12345) % (1 << 62), seed % (1 << 40)], dtype=torch.int64, device=dev)
    state["Y"] = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
    if case["op"].endswith("train"):
        state["dY"] = normal(m, n, 1.0)
        state["dX"] = torch.empty_like(state["X"])
        state["dA"] = torch.empty_like(state["A"])
        state["dB"] = torch.empty_like(state["B"])
    return state


# ------------------------------------------------------------ plain forms ----

def _exponent(amax):
    """The smallest e with amax <= 448 * 2**e, at least -127; 0 for an empty group."""
    mant, ex = torch.frexp(amax)                       # amax = mant * 2**ex, mant in [0.5, 1)
    e = torch.where(mant <= 0.875, ex - 9, ex - 8).clamp_min(-127)
    return torch.where(amax == 0, torch.zeros_like(e), e)


def _quantize(W):
    """(e4m3 codes, e8m0 scales) of W with one scale for each 128 x 128 block."""
    n, k = W.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    pad = torch.zeros(nb * BLOCK, kb * BLOCK, dtype=torch.float32, device=W.device)
    pad[:n, :k] = W.float()
    e = _exponent(pad.abs().view(nb, BLOCK, kb, BLOCK).amax(dim=(1, 3)))
    step = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    q = (pad.view(nb, BLOCK, kb, BLOCK) / step[:, None, :, None]).reshape(nb * BLOCK, kb * BLOCK)[:n, :k]
    return q.to(torch.float8_e4m3fn).contiguous(), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _weight(Wq, Ws):
    """The fp32 values that the codes and scales of an 8-bit weight stand for."""
    n, k = Wq.shape
    step = torch.ldexp(torch.ones(Ws.shape, device=Wq.device), Ws.view(torch.uint8).int() - 127)
    full = step.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return Wq.float() * full


def _rows(X):
    """The fp32 values of X rounded to e4m3 with one scale for each row and 128 columns."""
    m, k = X.shape
    kb = -(-k // BLOCK)
    pad = torch.zeros(m, kb * BLOCK, dtype=torch.float32, device=X.device)
    pad[:, :k] = X.float()
    e = _exponent(pad.abs().view(m, kb, BLOCK).amax(dim=2))
    step = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)[:, :, None]
    return ((pad.view(m, kb, BLOCK) / step).to(torch.float8_e4m3fn).float() * step).view(m, kb * BLOCK)[:, :k]


_LOW = 0xFFFFFFFF


def _philox_round(state, i):
    """One Philox4x32 round on int64 tensors that hold 32-bit words."""
    c0, c1, c2, c3, k0, k1 = state
    a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57              # the signed product's 64 bits are the unsigned one's
    key0, key1 = (k0 + i * 0x9E3779B9) & _LOW, (k1 + i * 0xBB67AE85) & _LOW
    return ((b >> 32) & _LOW) ^ c1 ^ key0, b & _LOW, ((a >> 32) & _LOW) ^ c3 ^ key1, a & _LOW, k0, k1


def _keep(rng, m, k, p):
    """(mask of the kept elements [m, k], 1 / the share that is kept)."""
    dev = rng.device
    c0 = torch.arange(k // 8, device=dev)[None, :].expand(m, -1)
    c1 = torch.arange(m, device=dev)[:, None].expand(-1, k // 8)
    seed, offset = rng[0], rng[1]
    start = (c0, c1, (offset & _LOW).expand(m, k // 8), ((offset >> 32) & _LOW).expand(m, k // 8),
             seed & _LOW, (seed >> 32) & _LOW)
    w = torch.stack(functools.reduce(_philox_round, range(7), start)[:4], dim=-1)
    lanes = torch.stack((w & 0xFFFF, w >> 16), dim=-1).reshape(m, k)
    t = math.floor(p * 65536.0 + 0.5)
    return lanes >= t, 65536.0 / (65536.0 - t)


def _plain(state):
    case = state["case"]
    op = case["op"]
    if op == "quantize":
        Wq, Ws = _quantize(state["W"])
        return {"W": _weight(Wq, Ws).bfloat16(), "exponents": Ws.view(torch.uint8)}
    m, k, p, s = case["M"], case["d_in"], case["p"], case["scale"]
    fp8 = op.startswith("fp8")
    X, A, B = state["X"].float(), state["A"].float(), state["B"].float()
    W = _weight(state["Wq"], state["Ws"]) if fp8 else state["W"].float()
    keep, up = _keep(state["rng"], m, k, p) if p > 0 else (None, 1.0)
    drop = (lambda t: torch.where(keep, t, 0.0) * up) if p > 0 else (lambda t: t)
    Xd = drop(X)
    T = s * (Xd @ A.T)
    out = {"Y": ((_rows(state["X"]) if fp8 else X) @ W.T + T @ B.T).bfloat16()}
    if op.endswith("train"):
        dY = state["dY"].float()
        dT = s * (dY @ B)
        out["dB"] = (dY.T @ T).bfloat16()
        out["dA"] = (dT.T @ Xd).bfloat16()
        out["dX"] = ((_rows(state["dY"]) if fp8 else dY) @ W + drop(dT @ A)).bfloat16()
    return out


def run(state):
    if own:
        return _own(state)
    return _plain(state)


def _own(state):
    import lora_linear_layer_b200 as L

    case = state["case"]
    op = case["op"]
    if op == "quantize":
        L.lora_quantize_fp8(state["W"], state["Wq"], state["Ws"])
        L.lora_dequantize_fp8(state["Wq"], state["Ws"], state["out"])
        return {"W": state["out"], "exponents": state["Ws"].view(torch.uint8)}
    m, k, n, r, p, s = (case[x] for x in ("M", "d_in", "d_out", "r", "p", "scale"))
    X, A, B, Y = state["X"], state["A"], state["B"], state["Y"]
    rng = state["rng"] if p > 0 else None
    train = op.endswith("train")
    grads = (state["dY"], state["dX"], state["dA"], state["dB"]) if train else None
    if "ws" not in state:
        need = (L.lora_fp8_workspace_size if op.startswith("fp8") else L.lora_bwd_workspace_size)(m, k, n, r)
        state["ws"] = torch.empty(need, dtype=torch.uint8, device=X.device)
    ws = state["ws"]
    if op.startswith("fp8"):
        Wq, Ws = state["Wq"], state["Ws"]
        L.lora_fwd_fp8(X, Wq, Ws, A, B, Y, s, ws, p, rng)
        if train:
            L.lora_bwd_fp8(X, Wq, Ws, A, B, *grads, s, ws, p, rng, L.LORA_BWD_T_SAVED)
    else:
        W = state["W"]
        L.lora_fwd_dropout(X, W, A, B, Y, s, p, rng, ws)
        if train:
            L.lora_bwd_dropout(X, W, A, B, *grads, s, p, rng, ws, L.LORA_BWD_T_SAVED)
    out = {"Y": Y}
    if train:
        out.update(dB=state["dB"], dA=state["dA"], dX=state["dX"])
    return out


# ------------------------------------------------------------ definition ----

def _grid(x, axis_blocks):
    """float64 values of x on the e4m3 grid of each block (a view [rows, rb, cols, cb] of x), and the exponents."""
    amax = x.abs().amax(dim=axis_blocks, keepdim=True)
    e = torch.ceil(torch.log2(amax.clamp_min(1e-300) / E4M3_MAX))
    # the logarithm is off by a rounding at most: settle it by the comparison itself
    e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= E4M3_MAX * torch.exp2(e - 1), e - 1, e).clamp_min(-127.0)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    v = x / torch.exp2(e)
    ulp = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / ulp) * ulp * torch.exp2(e)


def _blocked(x, rows):
    """x on the e4m3 grid, with one scale for each `rows` x 128 block."""
    m, k = x.shape
    mb, kb = -(-m // rows), -(-k // BLOCK)
    pad = torch.zeros(mb * rows, kb * BLOCK, dtype=torch.float64, device=x.device)
    pad[:m, :k] = x.double()
    return _grid(pad.view(mb, rows, kb, BLOCK), (1, 3)).reshape(mb * rows, kb * BLOCK)[:m, :k]


def _times(a, const):
    """(high, low) 32-bit words of a * const, by 16-bit halves."""
    al, ah, bl, bh = a % 65536, a // 65536, const % 65536, const // 65536
    mid = ah * bl + (al * bl) // 65536
    mid2 = al * bh + mid % 65536
    return ah * bh + mid // 65536 + mid2 // 65536, (al * bl) % 65536 + (mid2 % 65536) * 65536


def _kept(rng, m, k, p):
    """The mask by the definition, on host integers for the key and offset."""
    seed, offset = (int(v) for v in rng.tolist())
    dev = rng.device
    word = 1 << 32
    x = [torch.arange(k // 8, device=dev).repeat(m, 1), torch.arange(m, device=dev)[:, None].repeat(1, k // 8),
         torch.full((m, k // 8), offset % word, device=dev), torch.full((m, k // 8), offset // word % word, device=dev)]
    key = [seed % word, seed // word % word]
    rounds = 7
    while rounds:
        (h0, l0), (h1, l1) = _times(x[0], 0xD2511F53), _times(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % word, (key[1] + 0xBB67AE85) % word]
        rounds -= 1
    t = int(np.floor(p * 65536 + 0.5))
    halves = [h for w in x for h in (w % 65536, w // 65536)]
    return torch.stack(halves, dim=2).reshape(m, k) >= t, 1.0 / (1.0 - t / 65536)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return {"W": _blocked(state["W"], BLOCK), "exponents": None}
    X, A, B = state["X"].double(), state["A"].double(), state["B"].double()
    if op.startswith("fp8"):
        scale = torch.exp2(state["Ws"].view(torch.uint8).double() - 127)
        W = state["Wq"].double() * torch.kron(scale, torch.ones(BLOCK, BLOCK, dtype=torch.float64, device=X.device))[
            : case["d_out"], : case["d_in"]]
        Xb = _blocked(X, 1)
    else:
        W, Xb = state["W"].double(), X
    if case["p"] > 0:
        keep, up = _kept(state["rng"], case["M"], case["d_in"], case["p"])
        mask = keep.double() * up
    else:
        mask = torch.ones((), dtype=torch.float64, device=X.device)
    T = case["scale"] * ((mask * X) @ A.T)
    out = {"Y": Xb @ W.T + T @ B.T}
    if op.endswith("train"):
        dY = state["dY"].double()
        dT = case["scale"] * (dY @ B)
        out["dB"] = dY.T @ T
        out["dA"] = dT.T @ (mask * X)
        out["dX"] = (_blocked(dY, 1) if op.startswith("fp8") else dY) @ W + mask * (dT @ A)
    return out
