"""The model of the 8-bit paged cache where a block has a scale below 2^-126."""
import numpy as np
import pytest

from oracle import e4m3


@pytest.mark.parametrize("old", [2.0 ** -127, 1.5 * 2.0 ** -130, 2.0 ** -149])
@pytest.mark.parametrize("new", [0.0, 2.0 ** -149, 2.0 ** -130, 1e-38, 1.0])
def test_scales_below_the_least(old, new):
    """They give way to one whose reciprocal is finite; the older rows follow."""
    codes = np.full((1, 1, 16, 4), 0x7F, np.uint8)
    codes[0, 0, :2] = e4m3.encode(np.float32([[448, -2, 0, 1]] * 2))
    scales = np.float32([[old]])
    before = e4m3.gather(codes, scales, [0], 2)
    e4m3.append(codes, scales, [0], 2, np.full((1, 1, 4), new, np.float32))
    assert scales[0, 0] == max(e4m3.scale_for(np.float32(new)), np.float32(2.0 ** -126))
    got, step = e4m3.gather(codes, scales, [0], 3), float(scales[0, 0]) * 2.0 ** -10
    assert np.isfinite(got.numpy()).all()
    assert ((got[:, :2] - before).abs() <= before.abs() / 16 + step).all()
    assert ((got[:, 2] - np.float32(new)).abs() <= np.float32(new) / 16 + step).all()
