"""The pack's quotients: the product with the reciprocal times 1 + 2^-20, cut to 11 significant bits, modelled in binary32
with the NaN that a GPU's product gives (0x7FFFFFFF)."""
import numpy as np
import pytest
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float32)
ABOVE = np.float32(1 + 2.0 ** -20)


def near(x, inv):
    with np.errstate(over="ignore", invalid="ignore"):
        q = (x * inv).astype(np.float32)
    bits = np.where(np.isnan(q), np.uint32(0x7FFFFFFF), q.view(np.uint32))
    return (bits & np.uint32(0xFFFFE000)).view(np.float32)


def nearest(y, grid):
    """Index of the nearest, the even index on a tie."""
    mid = ((grid[1:].astype(np.float64) + grid[:-1]) / 2).astype(np.float32)
    lo, hi = np.searchsorted(mid, y, side="left"), np.searchsorted(mid, y, side="right")
    return np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))


@pytest.fixture(scope="module")
def e4m3():
    return torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()


def test_every_bf16_value_and_scale(e4m3):
    x = (np.arange(0x7F80, dtype=np.uint32) << 16).view(np.float32)          # every finite magnitude
    assert np.array_equal(nearest(near(x, ABOVE / np.float32(6)), e4m3), nearest(x / np.float32(6), e4m3))
    for s in e4m3[1:]:
        inv = np.float32(1) / s * ABOVE
        with np.errstate(over="ignore"):
            assert np.array_equal(nearest(near(x, inv), E2M1), nearest(x / s, E2M1)), s


def test_zeros_infinities_and_nan(e4m3):
    for s in e4m3[1:]:
        inv = np.float32(1) / s * ABOVE
        y = near(np.array([0.0, -0.0, np.inf, -np.inf, np.nan], np.float32), inv)
        assert np.array_equal(y[:4], [0.0, 0.0, np.inf, -np.inf]) and np.signbit(y[1]) and np.isnan(y[4]), s
