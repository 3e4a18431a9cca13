"""The 64-bit form of the 4-bit cache: pins of its roundings, ties and bytes."""
import numpy as np
import pytest

from oracle import kv4 as K


def test_scale_values():
    assert len(K.SCALES) == 127 and K.SCALES[0] == 0 and K.SCALES[1] == 2.0 ** -9 and K.SCALES[-1] == 448
    assert (np.diff(K.SCALES) > 0).all()


@pytest.mark.parametrize("x,value", [(0.25, 0), (0.26, 0.5), (0.75, 1), (1.25, 1), (1.75, 2), (2.5, 2), (2.51, 3), (3.5, 4),
                                     (5.0, 4), (5.01, 6), (-5.0, -4), (-0.75, -1)])
def test_codes_round_to_even_codes(x, value):
    row = np.zeros(16)
    row[0], row[5] = 6.0, x                 # a block maximum of 6: a scale of 1
    codes, scales = K.quantise(row, 1.0)
    assert K.SCALES[scales[0]] == 1 and K.values(codes, scales, 1.0)[5] == value


@pytest.mark.parametrize("top,scale", [(6 * 1.0625, 1.0), (6 * 1.1875, 1.25), (6 * 448 * 2, 448), (6 * 2.0 ** -10, 0),
                                       (6 * 2.0 ** -10 * 1.01, 2.0 ** -9), (0, 0)])
def test_scales_round_to_even_and_saturate(top, scale):
    row = np.zeros(16)
    row[3] = top
    for g in (1.0, 0.25, 2.0 ** 20):
        assert K.SCALES[K.quantise(row * g, g)[1][0]] == scale


def test_saturated_codes_and_blocks_that_are_not_finite():
    row = np.full((2, 32), 6.0)
    row[0, 0] = 1e30
    row[1, 17], row[1, 20] = np.inf, np.nan
    codes, scales = K.quantise(row, 1.0)
    v = K.values(codes, scales, 1.0)
    assert v[0, 0] == 6 * 448 and (v[0, 1:16] == 0).all() and (v[0, 16:] == 6).all()
    assert (v[1, :16] == 6).all() and np.isnan(v[1, 16:]).all() and scales[1, 1] == 0x7F


@pytest.mark.parametrize("d,page", [(16, 8), (48, 24), (80, 16), (128, 64)])
def test_bytes_there_and_back(d, page):
    rng = np.random.default_rng(d)
    codes, scales = rng.integers(0, 16, (page, d)), rng.integers(0, 127, (page, d // 16))
    mem = np.full(K.page_bytes(page, d), 0xFF, dtype=np.uint8)
    for t in range(page):
        K.put(mem, t, page, codes[t], scales[t])
    c, s = K.get(mem, page, d)
    assert (c == codes).all() and (s == scales).all()
    assert d % 32 == 0 or (mem == 0).sum() > 0


def test_every_value_is_exact_in_half_precision():
    codes = np.arange(16)[None, :].repeat(127, 0)
    v = K.values(codes, np.arange(127)[:, None], 1.0)
    assert (v == v.astype(np.float16)).all()
