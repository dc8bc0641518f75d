"""The packed store's error bounds as the header states them, at the smallest, the middle and the largest scales."""
import numpy as np
import pytest

from oracle import delta


@pytest.mark.parametrize("top", [2.0 ** -149, 1e-40, 2.0 ** -128, 1.5 * 2.0 ** -128, 63 * 2.0 ** -127,
                                 127.4 * 2.0 ** -127, 127.5 * 2.0 ** -127, 2.0 ** -119, 1.0, 127.5, 1e30,
                                 127.5 * 2.0 ** 121, float(np.finfo(np.float32).max)])
def test_restored_values(top):
    r = np.random.default_rng(7)
    x = (r.uniform(-1, 1, (50, 128)) * top).astype(np.float32).astype(np.float64)
    x[:, ::32] = np.float32(top)
    codes, scales = delta.pack(x)
    err = np.abs(delta.unpack(codes, scales) - x).reshape(50, 4, 32).max(-1)
    s = scales.astype(int)
    half = np.ldexp(1.0, s - 128)
    held = top > 127.5 * 2.0 ** 121
    assert ((s == 248) | ~np.array(held)).all()
    assert (err < 2 * half).all() if held else (err <= half).all()
    assert (err[s > 0] <= top / 127).all()
    assert ((s == 0) == (top < 127.5 * 2.0 ** -127)).all()
    if top <= 2.0 ** -128:
        assert (codes == 0).all()  # all of it is lost, as half of the smallest step is 2^-128


def test_the_relative_bound_needs_a_scale_above_the_smallest():
    """A block of tiny values may lose all of them: the bound at s = 0 is absolute."""
    x = np.full((1, 32), 1e-40)
    codes, scales = delta.pack(x)
    err = np.abs(delta.unpack(codes, scales) - x).max()
    assert scales[0, 0] == 0 and 1e-40 / 127 < err <= 2.0 ** -128
