"""The adapter with dropout and the 8-bit base in 64 bits, from their
definitions (numpy, CPU), and the error bounds of the kernels' outputs.
Shares no code with the library."""
from __future__ import annotations

import numpy as np

import oracle as O
import workloads as WL

HALF_BF16 = 2.0 ** -8     # a rounding to bf16 is off by at most this share of the value
HALF_FP32 = 2.0 ** -24
# an fp32 accumulation of n terms: each addition is off by at most one fp32
# step of the running sum, which is at most the sum of the magnitudes (a
# whole step, not half: the tensor cores may truncate when they align terms)
ACC = 2.0 * HALF_FP32


def f64(t) -> np.ndarray:
    return O.bf16_bits_to_f64(WL.bf16_bits(t.detach().cpu()))


# ------------------------------------------------------------- the mask ----

def philox(c0, c1, c2, c3, k0, k1, rounds=7):
    """Philox4x32 on uint64 arrays that hold 32-bit words."""
    u = np.uint64
    lo = u(0xFFFFFFFF)
    c0, c1, c2, c3 = (np.asarray(c, dtype=u) for c in (c0, c1, c2, c3))
    for _ in range(rounds):
        p0 = c0 * u(0xD2511F53)
        p1 = c2 * u(0xCD9E8D57)
        c0, c1, c2, c3 = (p1 >> u(32)) ^ c1 ^ u(k0), p1 & lo, (p0 >> u(32)) ^ c3 ^ u(k1), p0 & lo
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c0, c1, c2, c3


def threshold(p: float) -> int:
    return int(np.floor(np.float64(np.float32(p)) * 65536 + 0.5))


def keep_mask(seed: int, offset: int, M: int, K: int, p: float) -> np.ndarray:
    i, c = np.meshgrid(np.arange(M), np.arange(K // 8), indexing="ij")
    low = lambda v: int(v) & 0xFFFFFFFF
    words = philox(c, i, np.full_like(c, low(offset)), np.full_like(c, low(offset >> 32)), low(seed), low(seed >> 32))
    lanes = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], axis=-1)
    return lanes.reshape(M, K) >= threshold(p)


# --------------------------------------------------------- the 8-bit base ----

def e4m3_grid(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to even, for |v| <= 448."""
    ex = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    ulp = 2.0 ** (ex - 3)
    return np.rint(v / ulp) * ulp


def exponents(amax: np.ndarray) -> np.ndarray:
    """The smallest e >= -127 with amax <= 448 * 2**e; 0 where amax is 0."""
    e = np.full(amax.shape, -127, dtype=np.int64)
    for cand in range(-127, 121):
        e = np.where((amax > 448.0 * 2.0 ** e) & (e < cand + 1), cand + 1, e)
    return np.where(amax == 0, 0, e)


def _blocks(x, rb, cb):
    m, k = x.shape
    pad = np.zeros((-(-m // rb) * rb, -(-k // cb) * cb))
    pad[:m, :k] = x
    return pad.reshape(pad.shape[0] // rb, rb, pad.shape[1] // cb, cb)


def quantize(x: np.ndarray, rows: int):
    """(values on the grid, exponents) with one scale for each rows x 128 block."""
    b = _blocks(x, rows, 128)
    e = exponents(np.abs(b).max(axis=(1, 3)))
    s = 2.0 ** e[:, None, :, None].astype(np.float64)
    q = (e4m3_grid(b / s) * s).reshape(b.shape[0] * rows, -1)
    return q[:x.shape[0], :x.shape[1]], e


# ---------------------------------------------------------------- layers ----

def layer(X, W, A, B, scale, dY=None, mask=None, p=0.0, fp8=False):
    """{name: (value, bound)} of Y (and dX, dA, dB) for fp64 inputs; W is the
    base's values.  A bound adds, for each sum, ACC * (number of terms) *
    (sum of the terms' magnitudes), the bf16 rounding of the T and dT that go
    into the next product, and the output's own rounding."""
    scale = float(np.float32(scale))
    Xb = quantize(X, 1)[0] if fp8 else X
    up = 1.0 if mask is None else 65536.0 / (65536 - threshold(p))
    keep = 1.0 if mask is None else mask
    Xm = np.where(keep, X, 0.0) if mask is not None else X
    K, (N, r) = X.shape[1], B.shape
    absA, absB, absW = np.abs(A), np.abs(B), np.abs(W)

    def held(v, mag, n):   # a sum of n terms of magnitude `mag`, rounded to bf16 for the next product
        acc = (n + 2) * ACC * mag
        return acc + HALF_BF16 * (np.abs(v) + acc)

    def out(v, err):
        return v, err + HALF_BF16 * (np.abs(v) + err) + 2.0 ** -133

    T = scale * up * (Xm @ A.T)
    eT = held(T, abs(scale) * up * (np.abs(Xm) @ absA.T), K)
    mag = np.abs(Xb) @ absW.T + (np.abs(T) + eT) @ absB.T
    res = {"Y": out(Xb @ W.T + T @ B.T, eT @ absB.T + (K + r) * ACC * mag)}
    if dY is None:
        return res
    M = X.shape[0]
    dT = scale * (dY @ B)
    edT = held(dT, abs(scale) * (np.abs(dY) @ absB), N)
    tm = np.abs(T) + eT
    dm = np.abs(dT) + edT
    res["dB"] = out(dY.T @ T, np.abs(dY).T @ eT + (M + 2) * ACC * (np.abs(dY).T @ tm))
    res["dA"] = out(up * (dT.T @ Xm), up * (edT.T @ np.abs(Xm) + (M + 2) * ACC * (dm.T @ np.abs(Xm))))
    dYb = quantize(dY, 1)[0] if fp8 else dY
    low = up * np.where(keep, dT @ A, 0.0)
    elow = up * np.where(keep, edT @ absA + (r + 2) * ACC * (dm @ absA), 0.0)
    lowm = up * np.where(keep, dm @ absA, 0.0)
    res["dX"] = out(dYb @ W + low, elow + (N + r) * ACC * (np.abs(dYb) @ absW + lowm))
    return res


def check(name, got, ref):
    """`got` (numpy fp64) within ref = (value, bound), element for element."""
    v, bound = ref
    assert got.shape == v.shape, (name, got.shape, v.shape)
    err = np.abs(got - v)
    bad = ~(err <= bound)
    if bad.any():
        i = np.unravel_index(int(np.argmax(bad)), bad.shape)
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} outside the bound, first at {i}: "
                             f"{got[i]} for {v[i]} (bound {bound[i]}), worst ratio {np.nanmax(err / bound):.3g}")
    return float(np.max(err / bound)) if bad.size else 0.0
