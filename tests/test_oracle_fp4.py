"""The oracle of the 4-bit formats: tables, ties, blocks and the scales'
places (no GPU)."""
import numpy as np
import pytest

from oracle import fp4 as O


def test_the_tables():
    assert O.E4M3[1] == 2.0 ** -9 and O.E4M3[8] == 2.0 ** -6 and O.E4M3[126] == 448 and O.E4M3[0x38] == 1
    assert (np.diff(O.E4M3) > 0).all()
    code = np.arange(16)
    assert O.code_values(code).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6]


def test_ties_go_to_the_even_code():
    halves = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]
    assert O.MAGNITUDES[O.nearest(halves, O.MAGNITUDES)].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]
    for h in halves[:-1]:
        below, above = O.nearest([h - 1e-9, h + 1e-9], O.MAGNITUDES)
        assert above == below + 1


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_blocks(fmt):
    r = np.random.RandomState(1)
    x = r.randn(5, 128) * np.exp(r.randn(5, 1))
    c, s = O.quantize(x, fmt)
    v = O.values(c, s, fmt)
    d = np.repeat(O.scale_values(s, fmt), O.BLOCK[fmt], -1)
    u = np.abs(x) / d
    # half a step, or what saturates: NV's scale is at most 2^-4 below amax / 6,
    # MX's largest value is below 8 scales
    half = np.where(u < 2, 0.25, np.where(u < 4, 0.5, np.where(u <= 6, 1.0, u - 6)))
    assert (np.abs(v - x) <= half * d + 1e-15).all() and (u < (6.4 if fmt == "nvfp4" else 8)).all()
    # a block's own values come back
    c2, s2 = O.quantize(v, fmt)
    assert (O.values(c2, s2, fmt) == v).all()
    x[0, 3], x[2, 40] = np.nan, np.inf
    v = O.values(*O.quantize(x, fmt), fmt)
    n = O.BLOCK[fmt]
    assert np.isnan(v[0, :n]).all() and np.isfinite(v[0, n:]).all()
    assert np.isnan(v[2, 40 // n * n:40 // n * n + n]).all() and np.isfinite(v[1]).all()


def test_tensor_scale():
    assert O.tensor_scale([0.0, -0.0]) == 1 and O.tensor_scale([2688.0]) == 1 and O.tensor_scale([2689.0]) == 2
    assert O.tensor_scale([-1.0]) == 2.0 ** -11 and O.tensor_scale([np.nan, np.inf, 2688.0 * 8]) == 8
    for v in (1e-3, 0.07, 5.0, 1e5):
        t = O.tensor_scale([v])
        assert v <= 2688 * t < 2 * v


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("offsets", [[0, 1], [0, 5, 5, 300, 300, 301], [0, 127, 128, 256, 300, 557], [0, 128, 384]])
def test_no_two_scales_share_a_byte(fmt, offsets):
    for K in (64, 192, 256):
        at = O.scale_place(offsets, K, fmt)
        assert at.min() >= 0 and at.max() < O.scale_bytes(offsets[-1], len(offsets) - 1, K, fmt)
        assert np.unique(at).size == at.size
