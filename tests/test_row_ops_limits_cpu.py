"""Limits of the operators on feature rows that the host checks: nothing here reaches a
device, and the addresses are never read."""
import ctypes

import pytest

A, B, C = (0x10000000 * k for k in range(1, 4))  # aligned, far apart


@pytest.fixture(scope="module")
def sp():
    from submanifold_sparse_convolution_submconv3d_b200 import build as b
    b.build()
    import submanifold_sparse_convolution_submconv3d_b200 as p
    return p


def test_rope_frequencies_have_a_limit(sp):
    """From 2^64 on a double's steps hide the turn: refused, in a given list and in a ladder
    (base^(-9/10) of head_dim 64 is 2^64 at base 2^-71.1)."""
    for f in (2.0 ** 64, -2.0 ** 64, 1e299, float("inf"), float("nan")):
        for axis in (0, -1):
            with pytest.raises(sp.SpconvError, match="2\\^64"):
                sp.spconv_rope_create(4, freqs=[1.0, f], axes=[1, axis])
    for base in (2.0 ** -72, 1e-30, 1e-300, 5e-324):
        with pytest.raises(sp.SpconvError, match="2\\^64"):
            sp.spconv_rope_create(64, base=base)
    largest = 2.0 ** 64 - 2.0 ** 11
    for f in (largest, -largest, 0.0, 5e-324, -2.0 ** -1022):
        sp.spconv_rope_create(4, freqs=[1.0, f], axes=[1, 0]).free()
    for base in (2.0 ** -71, 1e-5, 0.5, 1.0, 1e299):
        sp.spconv_rope_create(64, base=base).free()
    sp.spconv_rope_create(10, base=5e-324).free()  # one pair an axis: base^0
