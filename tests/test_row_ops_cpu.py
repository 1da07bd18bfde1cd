"""Refusals of the operators on feature rows, none of which reaches a device: the C
entry points check sizes, alignment and overlap on the host, the binding shapes, types
and devices.  The addresses here are never read."""
import ctypes

import pytest

A, B, C, D, E = (0x10000000 * k for k in range(1, 6))  # aligned, far apart


@pytest.fixture(scope="module")
def sp():
    from submanifold_sparse_convolution_submconv3d_b200 import build as b
    b.build()
    import submanifold_sparse_convolution_submconv3d_b200 as p
    return p


def test_rms_norm_refusals(sp):
    def call(dtype=1, x=A, res=None, w=None, n=4, c=16, eps=1e-6, sum_out=None, out=B, rstd=None):
        return sp.lib.spconv_rms_norm(dtype, x, res, w, n, c, eps, sum_out, out, rstd, None)

    bad = [dict(dtype=2), dict(x=None), dict(n=-1), dict(n=1 << 31), dict(c=0), dict(c=65537), dict(eps=-1.0),
           dict(eps=float("nan")), dict(eps=float("inf")), dict(x=A + 4), dict(out=None), dict(out=B + 8), dict(w=C + 2),
           dict(rstd=D + 4), dict(out=A), dict(out=A + 112), dict(sum_out=C),                   # no residual
           dict(res=C, sum_out=C + 16), dict(res=C, sum_out=A + 16), dict(res=C, sum_out=B),    # partial overlaps
           dict(w=B), dict(rstd=A), dict(rstd=B + 16)]
    for kw in bad:
        assert call(**kw) == sp.INVALID_ARG, kw
        assert sp.lib.spconv_last_error(), kw
    assert call(n=0, x=None, out=None) == sp.OK


def test_rms_norm_q8_refusals(sp):
    def call(n=4, c=16, x=A, q=B, scale=C, sum_out=None, res=None):
        return sp.lib.spconv_rms_norm_q8(1, x, res, None, n, c, 1e-6, sum_out, q, scale, None)

    for kw in (dict(q=None), dict(scale=None), dict(q=B + 1), dict(scale=C + 4), dict(q=A), dict(scale=A),
               dict(scale=B), dict(res=D, sum_out=B)):
        assert call(**kw) == sp.INVALID_ARG, kw
    assert call(n=0, x=None) == sp.OK


def test_rms_norm_backward_refusals(sp):
    size = ctypes.c_int64()
    assert sp.lib.spconv_rms_norm_workspace(1000, 64, ctypes.byref(size)) == sp.OK and size.value > 0
    assert sp.lib.spconv_rms_norm_workspace(0, 64, ctypes.byref(size)) == sp.OK and size.value >= 0
    for n, c in ((-1, 64), (1 << 31, 64), (5, 0), (5, 65537)):
        assert sp.lib.spconv_rms_norm_workspace(n, c, ctypes.byref(size)) == sp.INVALID_ARG
    assert sp.lib.spconv_rms_norm_workspace(5, 5, None) == sp.INVALID_ARG

    def call(dy=A, h=B, w=None, rstd=C, dsum=None, n=4, c=16, dx=D, dw=None, ws=None):
        return sp.lib.spconv_rms_norm_backward(1, dy, h, w, rstd, dsum, n, c, dx, dw, ws, None)

    F = 0x60000000
    for kw in (dict(dy=None), dict(h=None), dict(rstd=None), dict(dx=None), dict(dx=A), dict(dx=B), dict(dx=C),
               dict(dsum=D + 16), dict(dy=A + 2), dict(dx=D + 8), dict(dw=E), dict(dw=E, ws=F + 4), dict(dw=E, ws=E),
               dict(dw=E, ws=A), dict(dw=D, ws=F), dict(dw=A, ws=F), dict(dw=E + 4, ws=F), dict(w=D), dict(n=-1),
               dict(c=0)):
        assert call(**kw) == sp.INVALID_ARG, kw
    assert call(n=0, dy=None, h=None, rstd=None, dx=None) == sp.OK


def test_rope_refusals(sp):
    handle = ctypes.c_void_p()
    dbl, i32 = lambda *v: (ctypes.c_double * len(v))(*v), lambda *v: (ctypes.c_int32 * len(v))(*v)

    def create(d=4, layout=0, base=1e4, freqs=None, axes=None, out=ctypes.byref(handle)):
        return sp.lib.spconv_rope_create(d, layout, base, freqs, axes, out)

    for kw in (dict(d=0), dict(d=3), dict(d=258), dict(layout=2), dict(base=0.0), dict(base=float("nan")),
               dict(freqs=dbl(1, 1)), dict(axes=i32(0, 0)), dict(freqs=dbl(1, float("inf")), axes=i32(0, 0)),
               dict(freqs=dbl(1, float("nan")), axes=i32(0, 0)), dict(freqs=dbl(1, 1), axes=i32(0, 3)),
               dict(freqs=dbl(1, 1), axes=i32(0, -2)), dict(out=None)):
        assert create(**kw) == sp.INVALID_ARG, kw
    assert handle.value is None
    assert sp.lib.spconv_rope_free(None) == sp.OK
    assert create(d=16, freqs=dbl(*[0.5] * 8), axes=i32(*[2] * 8)) == sp.OK

    def apply(rope=handle, dtype=1, coords=A, n=3, x=B, heads=2, xr=32, xh=16, out=C, outr=32, outh=16):
        return sp.lib.spconv_rope_apply(rope, dtype, coords, n, x, heads, xr, xh, out, outr, outh, 0, None)

    for kw in (dict(rope=None), dict(dtype=5), dict(coords=None), dict(coords=A + 4), dict(x=None), dict(out=None),
               dict(x=B + 1), dict(out=C + 1), dict(dtype=0, x=B + 2), dict(heads=0), dict(heads=4097), dict(n=-1),
               dict(n=1 << 31), dict(xr=15), dict(xh=8), dict(outr=8), dict(outh=-16), dict(xr=1 << 41),
               dict(outr=16, outh=16),        # rows and heads of out share elements
               dict(out=B, outr=64),          # in place with other strides
               dict(out=B + 32), dict(out=A)):
        assert apply(**kw) == sp.INVALID_ARG, kw
    assert apply(n=0, coords=None, x=None, out=None) == sp.OK
    assert sp.lib.spconv_rope_free(handle) == sp.OK


def test_w4_refusals(sp):
    lib = sp.lib
    F, G = 0x60000000, 0x70000000

    def lin(dtype=1, x=A, xs=None, n=2, cin=64, packed=B, s=C, z=D, group=64, bias=None, out=E, cout=8):
        return lib.spconv_linear_w4(dtype, x, xs, n, cin, packed, s, z, group, bias, out, cout, None)

    for kw in (dict(dtype=3), dict(x=None), dict(packed=None), dict(s=None), dict(z=None), dict(out=None), dict(n=-1),
               dict(cin=0), dict(cin=96), dict(cin=1 << 21), dict(cout=0), dict(cout=(1 << 20) + 1), dict(group=16),
               dict(group=0), dict(x=A + 8), dict(packed=B + 4), dict(bias=F + 2), dict(xs=F + 4), dict(out=A),
               dict(out=B + 16), dict(out=C), dict(bias=E), dict(xs=E)):
        assert lin(**kw) == sp.INVALID_ARG, kw
    assert lin(n=33) == sp.UNSUPPORTED and b"kernel size 1" in lib.spconv_last_error()
    assert lin(n=0, x=None, out=None) == sp.OK
    q = lambda w=A, packed=B, s=C, z=D, cin=64, cout=8, group=32: lib.spconv_w4_quantize(1, w, cin, cout, group, packed, s, z, None)
    for kw in (dict(w=None), dict(w=A + 2), dict(packed=A), dict(s=B), dict(z=C), dict(cin=40), dict(group=33)):
        assert q(**kw) == sp.INVALID_ARG, kw
    d = lambda w=A, packed=B, s=C, z=D: lib.spconv_w4_dequantize(1, packed, s, z, 64, 8, 32, w, None)
    for kw in (dict(w=None), dict(w=B), dict(w=C), dict(w=D), dict(packed=None)):
        assert d(**kw) == sp.INVALID_ARG, kw


def test_binding_refusals(sp):
    import torch

    assert sp.W4_MAX_ROWS == 32
    cpu = torch.zeros((4, 16), dtype=torch.bfloat16)
    for fn in (lambda: sp.spconv_rms_norm(cpu), lambda: sp.spconv_rms_norm_q8(cpu),
               lambda: sp.spconv_rms_norm_backward(cpu, cpu, None, torch.zeros(4)),
               lambda: sp.spconv_w4_quantize(torch.zeros((64, 8))), lambda: sp.spconv_w4_quantize(cpu[0]),
               lambda: sp.spconv_linear_w4(cpu, torch.zeros((8, 2), dtype=torch.int32), torch.zeros((8, 1)), torch.zeros((8, 1))),
               lambda: sp.spconv_rope_create(8, layout="other"), lambda: sp.spconv_rope_create(8, freqs=[1.0] * 4),
               lambda: sp.spconv_rope_create(8, freqs=[1.0] * 3, axes=[0] * 3)):
        with pytest.raises(ValueError):
            fn()
    with pytest.raises(sp.SpconvError):
        sp.spconv_rope_create(7)
    rope = sp.spconv_rope_create(8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sp.spconv_rope_apply(rope, torch.zeros((4, 4), dtype=torch.int32), torch.zeros((4, 2, 8)))
    sp.spconv_rope_free(rope)
    with pytest.raises(ValueError, match="freed"):
        sp.spconv_rope_apply(rope, torch.zeros((4, 4), dtype=torch.int32), torch.zeros((4, 2, 8)))
