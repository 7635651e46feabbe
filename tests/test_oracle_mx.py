"""Pins of the MX oracle (CPU): the format's printed values, the minimal
non-clipping scale, nearest rounding by brute force, and the bound of half a
step per element."""
import numpy as np
import pytest

from oracle import mx as omx


def test_grids():
    assert list(omx.GRID["fp4"]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    g = omx.GRID["fp8"]
    assert len(g) == 127 and g[-1] == 448 and g[1] == 2.0**-9 and g[8] == 2.0**-6
    assert (np.diff(g) > 0).all()


@pytest.mark.parametrize("fmt", omx.FORMATS)
def test_scale_is_the_smallest_that_clips_nothing(fmt):
    top = omx.GRID[fmt][-1]
    for amax in (top, np.nextafter(top, np.inf), top / 2, 1.0, 3.3e38, 1e-45, 2.0**-127 * top):
        X = np.zeros((1, 32))
        X[0, 5] = -amax
        _, s = omx.mx_quantize(X, fmt)
        e = int(s[0, 0]) - 127
        assert amax <= top * 2.0**e
        assert e == -127 or amax > top * 2.0 ** (e - 1)


@pytest.mark.parametrize("fmt", omx.FORMATS)
def test_nearest_with_ties_to_even_by_brute_force(fmt):
    grid = omx.GRID[fmt]
    mids = (grid[1:] + grid[:-1]) / 2
    x = np.concatenate([grid, mids, np.nextafter(mids, 0), np.nextafter(mids, 9e9)])
    x = np.concatenate([x, -x])
    x = np.pad(x, (0, -len(x) % 31)).reshape(-1, 31)
    x = np.concatenate([x, np.full((len(x), 1), grid[-1])], 1)  # scale 1 in every block
    codes, s = omx.mx_quantize(x, fmt)
    assert (s == 127).all()
    v = omx.mx_dequantize(codes, s, fmt, 32)
    for a, got in zip(np.abs(x).ravel(), np.abs(v).ravel()):
        d = np.abs(grid - a)
        best = np.flatnonzero(d == d.min())
        want = best[0] if len(best) == 1 else best[best % 2 == 0][0]
        assert got == grid[want]


@pytest.mark.parametrize("fmt", omx.FORMATS)
@pytest.mark.parametrize("cols", [1, 31, 32, 33, 100])
def test_round_trip_bound_and_idempotence(fmt, cols):
    rng = np.random.default_rng(3)
    X = rng.standard_normal((7, cols)) * np.exp2(rng.integers(-20, 20, (7, 1)))
    codes, s = omx.mx_quantize(X, fmt)
    assert codes.shape == (7, omx.padded(cols) // (2 if fmt == "fp4" else 1))
    v = omx.mx_dequantize(codes, s, fmt, cols)
    half = 2.0**-4 if fmt == "fp8" else 2.0**-2  # half a step relative to a normal element
    least = 2.0**-10 if fmt == "fp8" else 0.25    # half a subnormal step
    S = np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, 1)[:, :cols]
    assert (np.abs(v - X) <= np.maximum(half * np.abs(X), least * S)).all()
    assert np.array_equal(omx.mx_dequantize(*omx.mx_quantize(v, fmt), fmt, cols), v)


@pytest.mark.parametrize("fmt", omx.FORMATS)
def test_non_finite_blocks(fmt):
    X = np.ones((2, 64))
    X[0, 40] = np.inf
    X[1, 3] = np.nan
    codes, s = omx.mx_quantize(X, fmt)
    assert s[0, 1] == 255 and s[1, 0] == 255 and s[0, 0] != 255
    v = omx.mx_dequantize(codes, s, fmt, 64)
    assert np.isnan(v[0, 32:]).all() and np.isnan(v[1, :32]).all() and np.isfinite(v[0, :32]).all()
