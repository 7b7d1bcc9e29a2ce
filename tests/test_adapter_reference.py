"""The 64-bit reference of the dropout and 8-bit tests, against known answers
and by hand (CPU)."""
import numpy as np
import pytest
import torch

import adapter_reference as R


@pytest.mark.parametrize("rounds,ctr,key,want", [
    # the published known-answer vectors of Philox4x32
    (7, (0, 0, 0, 0), (0, 0), (0x5f6fb709, 0x0d893f64, 0x4f121f81, 0x4f730a48)),
    (7, (0xffffffff,) * 4, (0xffffffff,) * 2, (0x5207ddc2, 0x45165e59, 0x4d8ee751, 0x8c52f662)),
    (10, (0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
])
def test_philox_known_answers(rounds, ctr, key, want):
    got = R.philox(*(np.array([c]) for c in ctr), key[0], key[1], rounds=rounds)
    assert tuple(int(w[0]) for w in got) == want


@pytest.mark.parametrize("p", [0.05, 0.5, 0.9])
def test_mask_keeps_its_share(p):
    keep = R.keep_mask(3, 9, 512, 512, p)
    n = keep.size
    q = 1 - R.threshold(p) / 65536
    assert abs(keep.mean() - q) < 6 * (q * (1 - q) / n) ** 0.5
    other = R.keep_mask(3, 10, 512, 512, p)
    assert abs((keep == other).mean() - (q * q + (1 - q) ** 2)) < 6 * 0.5 / n ** 0.5


def test_e4m3_grid_is_the_cast():
    v = np.concatenate([np.linspace(-448, 448, 20001), 2.0 ** np.arange(-12.0, 9.0), [0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    want = torch.tensor(v, dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(R.e4m3_grid(v.astype(np.float32).astype(np.float64)), want)


def test_exponents_by_definition():
    amax = np.array([0.0, 448.0, 449.0, 447.0, 224.0, 225.0, 2.0 ** -140, 3.3e38, 1.0])
    e = R.exponents(amax)
    assert list(e[:6]) == [0, 0, 1, 0, -1, 0] and e[6] == -127 and 448 * 2.0 ** e[7] >= 3.3e38 > 448 * 2.0 ** (e[7] - 1)
    assert e[8] == -8
