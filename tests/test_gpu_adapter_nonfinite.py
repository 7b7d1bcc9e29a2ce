"""Infinities and NaN through the dropout and 8-bit layers, at sizes on both
sides of the border between the kernel that makes T for few tokens and the one
that does for many, and at ranks that are padded (8, 24, 40) and not (16)."""
import numpy as np
import pytest
import torch

import adapter_reference as R
from test_gpu_adapter_dropout import BF16, host, make, rng_tensor, run
from test_gpu_fp8 import quantized, run as run_fp8, values

pytestmark = pytest.mark.gpu

TOKENS = (64, 1100)
RANKS = (8, 16, 24, 40)


def check_with_non_finite(name, got, want, ref):
    """`want` says where the result is not finite, and what it is there; the
    rest lies within ref = (value, bound)."""
    there = ~np.isfinite(want)
    assert there.any()
    np.testing.assert_array_equal(got[there], want[there], err_msg=name)
    v, bound = (np.where(there, 0.0, a) for a in ref)
    R.check(name, np.where(there, 0.0, got), (v, bound))


def positive(t, *names):
    return dict(t, **{n: t[n].abs().clamp_min(2.0 ** -8) for n in names})


def reference(t, p, W=None, fp8=False):
    mask = R.keep_mask(1, 2, *t["X"].shape, p) if p else None
    with np.errstate(all="ignore"):
        return R.layer(R.f64(t["X"]), R.f64(t["W"]) if W is None else W, R.f64(t["A"]), R.f64(t["B"]), 1.0,
                       dY=R.f64(t["dY"]), mask=mask, p=p, fp8=fp8), mask


@pytest.mark.parametrize("p", [0.0, 0.5])
@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("M", TOKENS)
def test_an_infinity_of_x_stays_one(gpu, M, r, p):
    """With positive weights an infinite X[i, k] makes row i of Y infinite
    (not NaN), whether the adapter keeps the value or drops it; dB is infinite
    by dY's signs where it is kept, dA in column k by dT's."""
    K, N, row = 256, 192, M - 3
    t = positive(make(M, K, N, r), "W", "A", "B")
    mask = R.keep_mask(1, 2, M, K, p) if p else np.ones((M, K), dtype=bool)
    rng = rng_tensor(1, 2) if p else None
    for kept in (True, False) if p else (True,):
        k = int(np.flatnonzero(mask[row] == kept)[3])
        u = dict(t, X=t["X"].clone())
        u["X"][row, k] = float("inf")
        out = run(gpu, u, 1.0, p, rng)
        ref, _ = reference(u, p)
        Y = np.zeros((M, N))
        Y[row] = np.inf
        check_with_non_finite("Y", host(out["Y"]), Y, ref["Y"])
        R.check("dX", host(out["dX"]), ref["dX"])
        if kept:
            dB, dA = np.zeros((N, r)), np.zeros((r, K))
            dB[:] = np.copysign(np.inf, R.f64(u["dY"])[row])[:, None]
            dA[:, k] = np.copysign(np.inf, (R.f64(u["dY"]) @ R.f64(u["B"]))[row])
            np.testing.assert_array_equal(host(out["dB"]), dB)
            check_with_non_finite("dA", host(out["dA"]), dA, ref["dA"])
        else:
            for name in ("dB", "dA"):
                R.check(name, host(out[name]), ref[name])


@pytest.mark.parametrize("p", [0.0, 0.5])
@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("M", TOKENS)
def test_an_infinity_of_dy_stays_one(gpu, M, r, p):
    """The same for dY[i, n] and row i of dX."""
    K, N, row, n = 256, 192, M - 2, 77
    t = positive(make(M, K, N, r), "W", "A", "B")
    t["dY"][row, n] = float("inf")
    out = run(gpu, t, 1.0, p, rng_tensor(1, 2) if p else None)
    ref, _ = reference(t, p)
    dX = np.zeros((M, K))
    dX[row] = np.inf
    check_with_non_finite("dX", host(out["dX"]), dX, ref["dX"])
    R.check("Y", host(out["Y"]), ref["Y"])


@pytest.mark.parametrize("r", RANKS)
def test_dropped_values_are_gone_among_many_tokens(gpu, r):
    """Every dropped place of X holds an infinity or a NaN."""
    M, K, N = 1100, 264, 136
    t = make(M, K, N, r)
    t["W"].zero_()
    keep = torch.tensor(R.keep_mask(1, 2, M, K, 0.5))
    zero = torch.zeros((), dtype=BF16)
    bad = torch.where(torch.arange(M * K).view(M, K) % 3 == 0, float("nan"), float("inf")).to(BF16)
    ref, _ = reference(dict(t, X=torch.where(keep, t["X"], zero)), 0.5)
    out = run(gpu, dict(t, X=torch.where(keep, t["X"], bad)), 1.0, 0.5, rng_tensor(1, 2), saved=False)
    for name in ("dX", "dA", "dB"):
        R.check(name, host(out[name]), ref[name])


@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("M", TOKENS)
def test_non_finite_groups_over_an_8_bit_base(gpu, M, r):
    """A row of X with an infinity or a NaN makes that row of Y NaN, one of dY
    that row of dX; the other rows are what they were, bit for bit."""
    K, N = 512, 272
    t = make(M, K, N, r)
    base = quantized(gpu, t["W"])
    clean = run_fp8(gpu, t, base, 1.0)
    u = dict(t, X=t["X"].clone(), dY=t["dY"].clone())
    u["X"][M - 1, 300] = float("inf")
    u["X"][0, 5] = float("nan")
    u["dY"][M // 2, 270] = float("-inf")
    u["dY"][1, 0] = float("nan")
    got = run_fp8(gpu, u, base, 1.0)
    for name, rows in (("Y", [0, M - 1]), ("dX", [1, M // 2])):
        others = [i for i in range(M) if i not in rows]
        assert got[name][rows].isnan().all(), name
        assert torch.equal(got[name][others], clean[name][others]), name


@pytest.mark.parametrize("M", TOKENS)
def test_a_nan_block_of_an_8_bit_base(gpu, M):
    """An infinity in one 128 x 128 block of W makes that block's columns of Y
    (and of dX) NaN and leaves the others."""
    K, N, r = 272, 400, 24
    t = make(M, K, N, r)
    t["W"][130, 140] = float("inf")
    base = quantized(gpu, t["W"])
    out = run_fp8(gpu, t, base, 1.0)
    W = values(*base)
    W[128:256, 128:256] = 0.0
    ref, _ = reference(t, 0.0, W=W, fp8=True)
    for name in ("Y", "dX"):
        want = np.zeros(ref[name][0].shape)
        want[:, 128:256] = np.nan
        check_with_non_finite(name, host(out[name]), want, ref[name])
