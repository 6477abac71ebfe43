"""The model of the 8-bit paged cache where a row with an infinity or NaN comes and goes."""
import numpy as np
import pytest

from oracle import e4m3

D = 4


def _cache():
    return np.full((2, 1, 16, D), 0x7F, np.uint8), np.full((2, 1), -1, np.float32)


def _rows(n, seed=0):
    return np.random.default_rng(seed).normal(size=(n, 1, D)).astype(np.float32)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("first", [1, 7, 12])
@pytest.mark.parametrize("at", [0, 2])
def test_rows_before_a_bad_one_are_kept(bad, first, at):
    """A drafted row that is taken back leaves no trace, whether it is all or part of what was stored."""
    draft = _rows(4, 1)
    draft[at, 0, 2] = bad
    codes, scales = _cache()
    e4m3.append(codes, scales, [0, 1], 0, _rows(first))
    want = codes.copy(), scales.copy()
    e4m3.append(codes, scales, [0, 1], first, draft)
    assert np.isnan(scales[0, 0])
    # taken back as far as the bad row, or further
    for keep in range(at + 1):
        c, s = codes.copy(), scales.copy()
        e4m3.append(c, s, [0, 1], first + keep, _rows(2, 2))
        wc, ws = want[0].copy(), want[1].copy()
        e4m3.append(wc, ws, [0, 1], first, draft[:at])
        e4m3.append(wc, ws, [0, 1], first + keep, _rows(2, 2))
        assert s[0, 0] == ws[0, 0] and np.array_equal(c[0, :, :first + keep + 2], wc[0, :, :first + keep + 2])
    # behind it: not
    e4m3.append(codes, scales, [0, 1], first + at + 1, _rows(2, 2))
    assert np.isnan(scales[0, 0]) and (codes[0, 0, first + at:first + at + 3] == 0).all()
    e4m3.append(codes, scales, [0, 1], 0, _rows(1))
    assert scales[0, 0] == e4m3.scale_for(np.abs(_rows(1)).max())


def test_scales_that_are_no_power_of_two():
    """The rows before go to the next one; a NaN of another kind keeps none."""
    codes, scales = _cache()
    e4m3.append(codes, scales, [0, 1], 0, _rows(5))
    scales[0] *= np.float32(1.25)
    before, step = e4m3.gather(codes, scales, [0], 5), float(scales[0, 0])
    e4m3.append(codes, scales, [0, 1], 5, np.full((1, 1, D), np.nan, np.float32))
    e4m3.append(codes, scales, [0, 1], 5, 0.1 * _rows(1))
    assert scales[0, 0] == 2 * step / 1.25
    after = e4m3.gather(codes, scales, [0], 5)
    assert ((after - before).abs() <= before.abs() / 16 + float(scales[0, 0]) * 2.0 ** -10).all()
    for bits in (0x7FFFFFFF, 0x7FC00000, 0xFFC00000, 0x7FC00FFF):
        scales.view(np.uint32)[0, 0] = bits
        e4m3.append(codes, scales, [0, 1], 5, _rows(1))
        assert np.isnan(scales[0, 0])
