"""Limits of the operators on feature rows that the host checks: nothing here reaches a
device, and the addresses are never read."""
import ctypes

import pytest

A, B, C = (1 << k for k in (30, 42, 44))  # aligned, far apart


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


def test_rope_spans_past_64_bits_are_refused(sp):
    """2^24 steps of 2^40 elements are 2^64: the spans of x and out are not taken modulo that."""
    handle = ctypes.c_void_p()
    assert sp.lib.spconv_rope_create(16, 0, 1e4, None, None, ctypes.byref(handle)) == sp.OK

    def apply(n, xr, outr, heads=1, x=B, out=C):
        return sp.lib.spconv_rope_apply(handle, 1, A, n, x, heads, xr, 16, out, outr, 16, 0, None)

    for n, xr, outr in (((1 << 24) + 1, 16, 1 << 40), ((1 << 24) + 1, 1 << 40, 16), ((1 << 23) + 1, 1 << 40, 1 << 40),
                        ((1 << 31) - 1, 1 << 32, 1 << 32), ((1 << 24) + 1, 1 << 35, 1 << 35)):
        assert apply(n, xr, outr) == sp.INVALID_ARG, (n, xr, outr)
        assert b"2^57" in sp.lib.spconv_last_error()
        assert apply(n, xr, outr, heads=2) == sp.INVALID_ARG
    assert apply(0, 1 << 40, 1 << 40) == sp.OK
    assert sp.lib.spconv_rope_free(handle) == sp.OK


def test_column_bound_shows_a_lost_share():
    """The bound on the weight's gradient is tight enough that the rows of one of 148 CTAs,
    left out of the 64-bit sums, or a single row, show in most columns
    (a product 3 a b of two normals is under 0.41, the largest bound here, one time in four)."""
    import torch

    import row_ops_bounds as bounds

    g = torch.Generator().manual_seed(0)
    for n, c, item, per_thread in ((90001, 17, 8, 16), (80000, 24, 8, 16), (40000, 53, 4, 8), (50001, 130, 8, 16), (1500, 3333, 4, 8)):
        terms = torch.randn((n, c), generator=g, dtype=torch.float64) * 3 * torch.randn((n, c), generator=g, dtype=torch.float64)
        tol = bounds.column_bound(n, c, item, per_thread) * terms.abs().sum(0)
        rows = bounds.row_groups(c, item, per_thread)
        cta = (torch.arange(n) // rows) % 148
        for lost in (cta == 77, torch.arange(n) == 147 * rows):
            assert (terms[lost].sum(0).abs() > tol).double().mean() > 0.5, (n, c)
