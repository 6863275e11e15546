"""The reference of the MXFP4 operators itself: worked examples, and the
relations that its bounds rest on."""
import numpy as np
import pytest

from tests import mx_reference as R


def test_worked_block():
    """A block whose largest magnitude is 6: scale 1, every rounding and tie by hand."""
    x = np.zeros((1, 32))
    x[0, :16] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 0.26, 2.51, 3.49, 5.01, -0.0]
    nib, byte = R.quantize(x)
    assert byte[0, 0] == 127
    assert list(nib[0, 0, :16]) == [7, 15, 0, 2, 2, 4, 4, 6, 6, 8, 14, 1, 5, 5, 7, 8]
    codes, scales = R.pack(nib, byte)
    assert codes[0, 0] == 7 | 15 << 4 and list(scales[0]) == [127, 127, 127, 127]


@pytest.mark.parametrize("amax,byte", [(0.0, 0), (1.0, 125), (3.99, 126), (4.0, 127), (7.99, 127), (8.0, 128),
                                       (2.0 ** -149, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (3e38, 252),
                                       (np.inf, 255), (np.nan, 255)])
def test_exponent_byte(amax, byte):
    assert R.quantize(np.full((1, 5), amax))[1][0, 0] == byte


def test_values_invert_pack_and_rounding_is_idempotent():
    x = np.random.default_rng(0).normal(size=(7, 101)) * 2.0 ** np.random.default_rng(1).integers(-20, 20, (7, 101))
    once = R.rounded(x)
    assert np.array_equal(R.rounded(once), once) or np.abs(R.rounded(once) - once).max() == 0
    block = np.abs(R.pad_blocks(x)).max(-1, keepdims=True)
    assert (np.abs(R.pad_blocks(once) - R.pad_blocks(x)) <= block / 4).all()  # half the widest step, or 8 -> 6


def test_bounds_accept_the_reference_and_refuse_a_shifted_result():
    rng = np.random.default_rng(2)
    x, w = R.rounded(rng.normal(size=(5, 96))), R.rounded(rng.normal(size=(40, 96)))
    y, err = R.matmul(x, w, rng.normal(size=40), "silu")
    R.assert_close(y.astype(np.float32), y, err)
    codes, scales = R.pack(*R.quantize(y))
    R.assert_mx_close(codes, scales, y, err)
    with pytest.raises(AssertionError):
        R.assert_close(y + 1e-3, y, err)
    wrong = codes.copy()
    wrong[2, 3] ^= 1
    with pytest.raises(AssertionError):
        R.assert_mx_close(wrong, scales, y, err)


def test_norm_formulas():
    v = np.array([[3.0, 4.0], [0.0, 0.0]])
    assert np.allclose(R.norm(v, 0 * v, "rms", None, None, 0.5)[0][0], v[0] / np.sqrt(13.0))
    assert np.allclose(R.norm(v, 0 * v, "layer", [2.0, 2.0], [1.0, 1.0], 0.75)[0], [[0.0, 2.0], [1.0, 1.0]])
