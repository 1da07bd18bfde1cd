"""The operators on feature rows (RMS norm, rotary positions, 4-bit linear layer) on
the GPU against their 64-bit definitions, with the bounds of ``row_ops_ref``."""
import numpy as np
import pytest
import torch

import row_ops_ref as ref
from row_ops_ref import U, chain, rounding

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
DTYPES = [BF, F32]


@pytest.fixture(scope="module")
def sp():
    import submanifold_sparse_convolution_submconv3d_b200 as p
    return p


def randn(*shape, seed=0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def within(got, want, tol, what=""):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(),
                           float(((got.double() - want).abs() / tol.clamp(min=1e-300)).max()))


# ------------------------------------------------------------------ RMS norm

NORM_SIZES = [(1, 1), (1, 16), (3, 7), (5, 8), (2, 31), (7, 33), (64, 64), (33, 100), (1, 1024), (130, 128), (9, 256),
              (1000, 72), (3, 1000), (4, 2048), (2, 2050), (5, 4096), (3, 4104), (2, 8192), (2, 8200), (1, 16384),
              (2, 20000), (1, 32776), (1, 40001), (1, 65536), (2, 65535),
              (70, 24), (31, 80), (9, 90), (33, 144), (17, 320), (9, 700), (7, 696), (2500, 1400), (5, 6001), (3, 12001)]


def norm_inputs(n, c, dtype, residual, weight, seed=0):
    x = randn(n, c, seed=seed, dtype=dtype) * 3
    r = randn(n, c, seed=seed + 1, dtype=dtype) if residual else None
    w = (1 + 0.3 * randn(c, seed=seed + 2)).to(dtype) if weight else None
    return x, r, w


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,c", NORM_SIZES)
def test_rms_norm(sp, n, c, dtype):
    for residual, weight in ((False, True), (True, True), (True, False), (False, False)):
        x, r, w = norm_inputs(n, c, dtype, residual, weight)
        rstd = torch.empty(n, device="cuda")
        got = sp.spconv_rms_norm(x, w, residual=r, eps=1e-5, rstd=rstd)
        out, total = got if residual else (got, None)
        y, h, rs = ref.rms_norm(x, w, r, 1e-5)
        within(out, y, rounding(y, dtype) + chain(c) * U * y.abs(), "out")
        within(rstd, rs, chain(c) * U * rs, "rstd")
        if residual:
            within(total, h, rounding(h, dtype) + U * h.abs(), "sum")


def check_q8(q, scale, y, c):
    s = y.abs().amax(1) / 448
    within(scale, s, (chain(c) + 4) * U * s, "scale")
    v = y / scale.double()[:, None]
    # half a step: 2^-4 of a normal value, 2^-10 under 2^-6; a value next to the middle may fall either way
    step = torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10))
    within(q.float(), v, step + (chain(c) + 4) * U * v.abs(), "q")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,c", NORM_SIZES)
def test_rms_norm_q8(sp, n, c, dtype):
    for residual in (False, True):
        x, r, w = norm_inputs(n, c, dtype, residual, True, seed=5)
        got = sp.spconv_rms_norm_q8(x, w, residual=r, eps=1e-5)
        y, h, _ = ref.rms_norm(x, w, r, 1e-5)
        assert got[0].dtype == torch.float8_e4m3fn and got[0].shape == (n, c)
        check_q8(got[0], got[1], y, c)
        if residual:
            within(got[2], h, rounding(h, dtype) + U * h.abs(), "sum")


@pytest.mark.parametrize("c", [48, 333, 4096])
def test_rms_norm_in_place_sum_and_unaligned_inputs(sp, c):
    x, r, w = norm_inputs(11, c, BF, True, True)
    y, h, _ = ref.rms_norm(x, w, r, 1e-6)
    want = sp.spconv_rms_norm(x, w, residual=r)
    for target in ("residual", "x"):
        a, b = x.clone(), r.clone()
        out, total = sp.spconv_rms_norm(a, w, residual=b, sum_out=b if target == "residual" else a)
        assert total is (b if target == "residual" else a)
        assert torch.equal(out, want[0]) and torch.equal(total, want[1])
        a, b = x.clone(), r.clone()
        q = sp.spconv_rms_norm_q8(a, w, residual=b, sum_out=b if target == "residual" else a)
        assert torch.equal(q[2], want[1])
        check_q8(q[0], q[1], y, c)
    wide = torch.empty((11, c + 3), dtype=BF, device="cuda")
    wide[:, 1:c + 1] = x
    odd = torch.empty(11 * c + 1, dtype=BF, device="cuda")[1:].view(11, c)  # off the 16-byte grid
    odd.copy_(r)
    got = sp.spconv_rms_norm(wide[:, 1:c + 1], w, residual=odd)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("c", [64, 65, 8192])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rms_norm_special_rows(sp, c, dtype):
    x = randn(8, c, dtype=dtype)
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] *= 1e-30
    x[4] = 0
    x[4, 7] = 1e-38
    x[5] *= 1e15
    w = torch.ones(c, dtype=dtype, device="cuda")
    out = sp.spconv_rms_norm(x, w, eps=1e-6)
    q, s = sp.spconv_rms_norm_q8(x, w, eps=1e-6)
    y, _, _ = ref.rms_norm(x, w, None, 1e-6)
    keep = [0, 3, 4, 5, 6, 7]
    within(out[keep], y[keep], rounding(y[keep], dtype) + chain(c) * U * y[keep].abs() + 1e-37)
    assert (out[0] == 0).all() and (q[0].float() == 0).all() and float(s[0]) == 2.0 ** -126
    # an infinite element: 1 / rms = 0, so inf * 0 there and 0 elsewhere, as the formula gives in fp32
    assert out[1, 3].isnan() and (out[1, :3] == 0).all() and (out[1, 4:] == 0).all()
    assert out[2].isnan().all()
    assert s[1].isnan() and s[2].isnan() and q[1].float().isnan().all() and q[2].float().isnan().all()
    # the tiny rows keep their values (scale at least 2^-126)
    v = y[[3, 4]] / s[[3, 4]].double()[:, None]
    within(q[[3, 4]].float(), v, torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) * 1.001)
    bad = sp.spconv_rms_norm(torch.zeros((2, c), dtype=dtype, device="cuda"), w, eps=0.0)
    assert bad.isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,c", [(1, 1), (2, 5), (3, 16), (257, 24), (1025, 128), (700, 100), (5000, 64), (33, 1024),
                                 (20, 2048), (17, 2056), (9, 4096), (3, 8192), (5, 8200), (2, 16384), (3, 20001),
                                 (2, 32776), (1, 65536),
                                 # several turns of every CTA
                                 (60000, 40), (50001, 130), (6000, 515), (3000, 1001), (1700, 4096), (700, 8192), (900, 12000),
                                 (90001, 17), (80000, 24), (40000, 53), (9000, 163), (4000, 932), (1500, 3333), (900, 4104),
                                 (1000, 5491), (500, 9001), (4, 2301), (5, 7000)])
def test_rms_norm_backward(sp, n, c, dtype):
    for weight, dsum in ((True, False), (True, True), (False, True)):
        h, d, w = norm_inputs(n, c, dtype, dsum, weight, seed=9)
        dy = randn(n, c, seed=12, dtype=dtype)
        rstd = ref.rms_norm(h, None, None, 1e-6)[2].float()
        dx, dw = sp.spconv_rms_norm_backward(dy, h, w, rstd, dsum=d)
        want, wantw, mag, magw = ref.rms_norm_backward(dy, h, w, rstd, d)
        within(dx, want, rounding(want, dtype) + (chain(c) + 4) * U * mag, "dx")
        if weight:
            within(dw, wantw, (n + 8) * U * magw, "dweight")
            again = sp.spconv_rms_norm_backward(dy, h, w, rstd, dsum=d)[1]
            assert torch.equal(dw, again), "the same inputs give the same bits"
            only = sp.spconv_rms_norm_backward(dy, h, w, rstd, dsum=d, weight_grad=False)
            assert only[1] is None and torch.equal(only[0], dx)
        else:
            assert dw is None
        if dsum:
            inplace = d.clone()
            assert torch.equal(sp.spconv_rms_norm_backward(dy, h, w, rstd, dsum=inplace, dx=inplace)[0], dx)


def test_rms_norm_backward_against_autograd_and_differences(sp):
    n, c, eps = 6, 40, 1e-6
    x, r, w = norm_inputs(n, c, F32, True, True, seed=20)
    dy, dh = randn(n, c, seed=21), randn(n, c, seed=22)
    rstd = torch.empty(n, device="cuda")
    _, h = sp.spconv_rms_norm(x, w, residual=r, eps=eps, rstd=rstd)
    dx, dw = sp.spconv_rms_norm_backward(dy, h, w, rstd, dsum=dh)

    def loss(a, b):
        t = a + r.double()
        return ((t * torch.rsqrt((t * t).mean(1, keepdim=True) + eps) * b) * dy.double()).sum() + (t * dh.double()).sum()

    a, b = x.double().requires_grad_(), w.double().requires_grad_()
    ga, gb = torch.autograd.grad(loss(a, b), (a, b))
    # h and rstd are rounded to fp32 before the gradient reads them: some 2^-24 of each term
    _, _, mag, magw = ref.rms_norm_backward(dy, h, w, rstd, dh)
    within(dx, ga, (chain(c) + 8) * U * mag + U * ga.abs())
    within(dw, gb, (n + 12) * U * magw)
    # central differences in 64 bits, step 1e-5: the truncation is far under the fp32 bound
    for (i, j) in ((0, 0), (2, 17), (5, 39)):
        e = torch.zeros((n, c), dtype=torch.float64, device="cuda")
        e[i, j] = 1e-5
        num = float(loss(x.double() + e, w.double()) - loss(x.double() - e, w.double())) / 2e-5
        assert abs(num - float(dx[i, j])) <= 1e-6 + 64 * U * float(mag[i, j])
        num = float(loss(x.double(), w.double() + e[i]) - loss(x.double(), w.double() - e[i])) / 2e-5
        assert abs(num - float(dw[j])) <= 1e-6 + 64 * U * float(magw[j])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,c", [(9, 3), (40, 17), (2001, 36), (700, 57), (700, 61), (301, 125), (301, 130), (150, 250),
                                 (150, 500), (77, 1018), (5, 2047), (40, 2047), (9, 2301), (30, 4091), (7, 5491),
                                 (9, 8186), (10, 16381), (6, 32765), (6, 32767)])
def test_rms_norm_rows_that_start_anywhere(sp, n, c, dtype):
    """Rows that begin and end inside an item of 16 bytes: every start, first and last rows, and
    neighbours of infinities and NaN that must not reach the row; nothing is written around them."""
    x, r, w = norm_inputs(n, c, dtype, True, True, seed=c)
    x[n // 2] = float("nan")
    x[n // 3] = float("inf")
    keep = [i for i in range(n) if i not in (n // 2, n // 3)]
    y, h, rs = ref.rms_norm(x, w, r, 1e-5)
    around = torch.full((n * c + 64,), 5.0, dtype=dtype, device="cuda")
    out = around[32:32 + n * c].view(n, c)
    sp.spconv_rms_norm(x, w, residual=r, eps=1e-5, out=out)
    within(out[keep], y[keep], rounding(y[keep], dtype) + chain(c) * U * y[keep].abs())
    q = torch.full((n * c + 64,), 5.0, device="cuda").to(torch.float8_e4m3fn)
    s = torch.empty(n, device="cuda")
    sp.spconv_rms_norm_q8(x, w, residual=r, eps=1e-5, out=q[32:32 + n * c].view(n, c), scale=s)
    check_q8(q[32:32 + n * c].view(n, c)[keep], s[keep], y[keep], c)
    # the gradient: a row of NaN and one of infinities stay in their rows of dx
    dy = randn(n, c, seed=3, dtype=dtype)
    d = randn(n, c, seed=4, dtype=dtype)
    hs = x.clone()
    hs[n // 3] = 1
    rstd = torch.ones(n, device="cuda")
    dback = around.clone()
    dx = dback[32:32 + n * c].view(n, c)
    for dsum in (None, d):
        sp.spconv_rms_norm_backward(dy, hs, w, rstd, dsum=dsum, dx=dx)
        want, _, mag, _ = ref.rms_norm_backward(dy, hs, w, rstd, dsum)
        rows = [i for i in range(n) if i != n // 2]
        within(dx[rows], want[rows], rounding(want[rows], dtype) + (chain(c) + 4) * U * mag[rows], "dx")
        assert dx[n // 2].isnan().all()
    for buf in (around, dback, q):
        assert (buf[:32].float() == 5).all() and (buf[32 + n * c:].float() == 5).all()
    # the weight's gradient over clean rows
    hs[n // 2] = 1
    _, dw = sp.spconv_rms_norm_backward(dy, hs, w, rstd)
    _, wantw, _, magw = ref.rms_norm_backward(dy, hs, w, rstd, None)
    within(dw, wantw, (n + 8) * U * magw, "dweight")


def test_rms_norm_empty(sp):
    z = torch.empty((0, 24), dtype=BF, device="cuda")
    w = torch.ones(24, dtype=BF, device="cuda")
    assert sp.spconv_rms_norm(z, w).shape == (0, 24)
    assert sp.spconv_rms_norm(z, w, residual=z)[1].shape == (0, 24)
    assert sp.spconv_rms_norm_q8(z, w)[1].shape == (0,)
    dx, dw = sp.spconv_rms_norm_backward(z, z, w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 24) and (dw == 0).all()


# ------------------------------------------------------------------ rotary positions

def rope_tol(want, mag, dtype):
    """fp32: the fraction of a turn rounded to fp32 (pi 2^-25), sincospif (2 ulp, 2^-23),
    three roundings of the products and their sum: under 2^-21 of |a| + |b|.  bf16 may
    use the fast sine and cosine, which are off by up to 2^-21.2 on [-pi, pi]: 2^-20."""
    return rounding(want, dtype) + mag * (2.0 ** -20 if dtype == BF else 2.0 ** -21)


def coords_for(n, extent, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, extent, (n, 4), generator=g, device="cuda", dtype=torch.int64)
    if extent > 1:
        c[-1, 1:] = extent - 1
    c[:, 0] = 1
    return c.to(torch.int32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("n,heads,d", [(1, 1, 2), (1, 16, 64), (2, 3, 6), (5, 2, 10), (33, 1, 64), (17, 5, 96), (64, 12, 64),
                                       (9, 8, 128), (7, 3, 80), (3, 4, 256), (1000, 2, 32), (31, 7, 20), (3, 65, 16), (2, 4096, 6),
                                       # several turns of every warp
                                       (30011, 5, 64), (20003, 12, 96), (40000, 1, 36)])
def test_rope(sp, n, heads, d, layout, dtype):
    x = randn(n, heads, d, dtype=dtype)
    freqs, axes = ref.rope_default(d)
    rope = sp.spconv_rope_create(d, layout=layout)
    for extent in (2, 512, 65536):
        coords = coords_for(n, extent, seed=d)
        for inverse in (False, True):
            want, mag = ref.rope(x, coords, freqs, axes, layout, inverse)
            got = sp.spconv_rope_apply(rope, coords, x, inverse=inverse)
            within(got, want, rope_tol(want, mag, dtype), (extent, inverse))
            y = x.clone()
            assert sp.spconv_rope_apply(rope, coords, y, out=y, inverse=inverse) is y and torch.equal(y, got)
    rope.free()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
@pytest.mark.parametrize("n,hq,hk,d", [(1, 4, 2, 64), (37, 6, 2, 64), (12, 5, 5, 24), (6, 3, 1, 30)])
def test_rope_in_a_packed_projection(sp, n, hq, hk, d, layout, dtype):
    """Queries and keys turned in place inside [n, (hq + 2 hk) d]; the values stay."""
    qkv = randn(n, (hq + 2 * hk) * d, dtype=dtype)
    before = qkv.clone()
    coords = coords_for(n, 300)
    rope = sp.spconv_rope_create(d, layout=layout)
    heads = qkv[:, :(hq + hk) * d].unflatten(1, (hq + hk, d))
    sp.spconv_rope_apply(rope, coords, heads, out=heads)
    want, mag = ref.rope(before[:, :(hq + hk) * d].unflatten(1, (hq + hk, d)), coords, *ref.rope_default(d), layout, False)
    within(heads, want, rope_tol(want, mag, dtype))
    assert torch.equal(qkv[:, (hq + hk) * d:], before[:, (hq + hk) * d:])
    # heads outside rows ([heads, n, d] memory), from one buffer into another with other strides
    t = before[:, :hq * d].unflatten(1, (hq, d)).transpose(0, 1).contiguous().transpose(0, 1)
    buf = torch.full((n + 2, hq + 1, d + 8), 7.0, dtype=dtype, device="cuda")
    out = buf[1:n + 1, :hq, 3:d + 3]
    sp.spconv_rope_apply(rope, coords, t, out=out)
    within(out, want[:, :hq], rope_tol(want[:, :hq], mag[:, :hq], dtype))
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[1:n + 1, :hq, 3:d + 3] = False
    assert (buf[mask] == 7).all()
    # a key shared by the heads (stride 0) is copied first
    one = before[:, None, :d].expand(n, 3, d)
    assert torch.equal(sp.spconv_rope_apply(rope, coords, one), sp.spconv_rope_apply(rope, coords, one.contiguous()))


@pytest.mark.parametrize("dtype", DTYPES)
def test_rope_own_frequencies_and_any_coordinate(sp, dtype):
    """One ladder cut into sections of time, height and width; negative and 32-bit extremes."""
    d, sections = 64, (8, 12, 12)
    freqs = [1e6 ** (-2 * j / d) for j in range(d // 2)]
    freqs[3], freqs[20] = -freqs[3], 40.0
    axes = [a for a, m in enumerate(sections) for _ in range(m)]
    axes[5] = -1
    rope = sp.spconv_rope_create(d, layout="halves", freqs=freqs, axes=axes)
    coords = torch.tensor([[0, 0, 0, 0], [0, -1, -7, -300], [5, 2 ** 31 - 1, -2 ** 31, 123456789], [0, 7, -65535, 40000],
                           [0, 1, 2, 3]], dtype=torch.int32, device="cuda")
    x = randn(5, 3, d, dtype=dtype)
    got = sp.spconv_rope_apply(rope, coords, x)
    want, mag = ref.rope(x, coords, freqs, axes, "halves", False)
    # the 64-bit reference itself rounds its angles: up to 2^31 * 40 rad * 2^-53
    far = torch.tensor([0, 0, 1, 0, 0], device="cuda").view(5, 1, 1) * (40 * 2.0 ** 31 * 2.0 ** -52)
    within(got, want, rope_tol(want, mag, dtype) + mag * far)
    assert torch.equal(got[0], x[0])
    back = sp.spconv_rope_apply(rope, coords, got.float(), inverse=True)
    within(back, x.double(), 2 * mag * 2.0 ** -20 + 2 * rounding(mag, dtype))


def test_rope_gradient_is_the_inverse(sp):
    n, heads, d = 4, 2, 16
    x, dy, coords = randn(n, heads, d), randn(n, heads, d, seed=1), coords_for(n, 1000)
    rope = sp.spconv_rope_create(d)
    dx = sp.spconv_rope_apply(rope, coords, dy, inverse=True)
    freqs, axes = ref.rope_default(d)
    loss = lambda a: float((ref.rope(a, coords, freqs, axes, "interleaved", False)[0] * dy.double()).sum())
    for at in ((0, 0, 0), (1, 1, 7), (3, 0, 15), (2, 1, 10)):
        e = torch.zeros((n, heads, d), dtype=torch.float64, device="cuda")
        e[at] = 1e-3  # the loss is linear in x: the difference is exact up to the sums' rounding
        num = (loss(x.double() + e) - loss(x.double() - e)) / 2e-3
        assert abs(num - float(dx[at])) <= 1e-9 + 4 * 2.0 ** -21 * float(dy[at[0], at[1]].abs().max())


def test_rope_empty(sp):
    rope = sp.spconv_rope_create(8)
    assert sp.spconv_rope_apply(rope, torch.empty((0, 4), dtype=torch.int32, device="cuda"),
                                torch.empty((0, 3, 8), device="cuda")).shape == (0, 3, 8)


# ------------------------------------------------------------------ 4-bit linear layer

def w4_inputs(cin, cout, group, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    packed = torch.randint(-2 ** 31, 2 ** 31, (cout, cin // 8), generator=g, device="cuda").to(torch.int32)
    s = (0.2 + torch.rand((cout, cin // group), generator=g, device="cuda")) * 0.1
    z = s * (-7.5 + torch.randn(s.shape, generator=g, device="cuda"))
    return packed, s.to(dtype), z.to(dtype)


def x8_inputs(n, cin, seed=0):
    x = randn(n, cin, seed=seed)
    s = x.abs().amax(1) / 448
    return (x / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), s


W4_SHAPES = [(32, 1, 32), (64, 8, 64), (128, 16, 128), (96, 5, 32), (160, 33, 32), (192, 64, 64), (256, 100, 64),
             (320, 129, 64), (384, 250, 128), (1024, 257, 64), (2048, 64, 128), (4096, 48, 32), (1504, 131, 32),
             (8192, 40, 128), (4160, 1030, 64),
             # several tiles a CTA and waves of CTAs, ragged; more groups than a CTA holds at a time
             (512, 9999, 64), (160, 19001, 32), (256, 40003, 128), (16416, 24, 32), (16448, 5003, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cin,cout,group", W4_SHAPES)
def test_linear_w4(sp, cin, cout, group, dtype):
    w = w4_inputs(cin, cout, group, dtype)
    bias = randn(cout, seed=3, dtype=dtype)
    for n in (1, 2, 3, 7, 8, 9, 15, 16, 17, 24, 25, 31, 32):
        x = randn(n, cin, seed=n, dtype=dtype) + (0.5 if n % 2 else 0)
        buf = torch.full((n + 3, cout), 9.0, dtype=dtype, device="cuda")
        sp.spconv_linear_w4(x, *w, bias=bias, out=buf[:n])
        want, err = ref.linear_w4(x, *w, bias, None)
        within(buf[:n], want, rounding(want, dtype) + err, n)
        assert (buf[n:] == 9).all(), "rows behind the last stay"
        q, s = x8_inputs(n, cin, seed=n)
        want, err = ref.linear_w4(q.float(), *w, None, s)
        within(sp.spconv_linear_w4(q, *w, x_scale=s), want, rounding(want, dtype) + err, n)


def test_linear_w4_rows_do_not_touch_each_other(sp):
    """A NaN row and an infinite row leave the others as they are; a result does not
    depend on which rows run with it (the sums of a row are its own)."""
    w = w4_inputs(512, 96, 64, BF)
    x = randn(12, 512, dtype=BF)
    clean = sp.spconv_linear_w4(x, *w)
    x[3, 100] = float("nan")
    x[7, 5] = float("inf")
    got = sp.spconv_linear_w4(x, *w)
    keep = [0, 1, 2, 4, 5, 6, 8, 9, 10, 11]
    assert torch.equal(got[keep], clean[keep])
    assert got[3].isnan().all() and not got[7].isfinite().any()


def test_linear_w4_extreme_codes(sp):
    """All codes 0, all 15, zero scales, zero rows, e4m3's largest values and NaN."""
    cin, cout = 256, 40
    x = randn(5, cin, dtype=F32)
    x[2] = 0
    for word in (0, -1, 0x0F0F0F0F, -0x0F0F0F10, 0x77777777):
        packed = torch.full((cout, cin // 8), word, dtype=torch.int32, device="cuda")
        s, z = randn(cout, 4, seed=1), randn(cout, 4, seed=2)
        s[0] = 0
        want, err = ref.linear_w4(x, packed, s, z, None, None)
        within(sp.spconv_linear_w4(x, packed, s, z), want, rounding(want, F32) + err)
    q = torch.full((3, cin), 448.0, device="cuda").to(torch.float8_e4m3fn)
    q.view(torch.uint8)[1] = 1     # the smallest value, 2^-9
    q.view(torch.uint8)[2, 9] = 127
    xs = torch.tensor([1.0, 2.0 ** -126, 1.0], device="cuda")
    w = w4_inputs(cin, cout, 64, F32)
    want, err = ref.linear_w4(q.float(), *w, None, xs)
    got = sp.spconv_linear_w4(q, *w, x_scale=xs)
    within(got[:2], want[:2], rounding(want[:2], F32) + err[:2] + 2.0 ** -126)
    assert got[2].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cin,cout,group", [(32, 1, 32), (64, 3, 64), (256, 70, 32), (384, 300, 128), (1024, 129, 64)])
def test_w4_quantize_and_back(sp, cin, cout, group, dtype):
    w = (randn(cin, cout, seed=4) * 0.05 + 0.01).to(dtype)
    w[:group, 0] = 0.25  # a constant group: scale 0, code 0
    packed, s, z = sp.spconv_w4_quantize(w, group)
    g, s_want, z_want = ref.w4_quantize(w, group)
    # (max - min) / 15 divided in fp32: the same quotient up to its last bit before the rounding
    assert torch.equal(z, z_want)
    within(s, s_want.double(), 2 * rounding(s_want.double(), dtype))
    q = ref.w4_codes(packed).view(cout, -1, group).double()
    sd, zd = s.double()[:, :, None], z.double()[:, :, None]
    at = torch.where(sd > 0, (g - zd) / sd.clamp(min=1e-300), torch.zeros_like(g))
    nearest = at.clamp(0, 15)
    assert ((q - nearest).abs() <= 0.5 + 64 * U * (1 + at.abs())).all()
    assert (q[0, 0] == 0).all() and float(s[0, 0]) == 0
    back = sp.spconv_w4_dequantize(packed, s, z)
    want = (q * sd + zd).flatten(1).t()
    assert back.shape == (1, cin, cout)
    within(back[0], want, rounding(want, dtype) + 2 * U * (q * sd + zd.abs()).flatten(1).t())
    again = sp.spconv_w4_quantize(back, group)
    assert again[0].shape == packed.shape


def test_linear_w4_against_the_kernel_size_1_layer(sp):
    """The same weights unpacked and run as a layer of kernel size 1."""
    cin, cout, n = 256, 128, 32
    packed, s, z = sp.spconv_w4_quantize((randn(1, cin, cout) * cin ** -0.5).to(BF), 64)
    bias, x = randn(cout, seed=1, dtype=BF), randn(n, cin, seed=2, dtype=BF)
    coords = torch.zeros((n, 4), dtype=torch.int32, device="cuda")
    coords[:, 3] = torch.arange(n)
    m = sp.spconv_build_map(coords, (1, 1, n), 1)
    layer = sp.spconv_subm_forward(m, x, sp.spconv_w4_dequantize(packed, s, z), bias)
    m.free()
    got = sp.spconv_linear_w4(x, packed, s, z, bias=bias)
    # the layer's weights are rounded to bf16: 2^-8 of each product, and either result's rounding
    w = ref.linear_w4(x.abs(), packed, s.abs(), z.abs(), None, None)[0]
    within(got, layer.double(), w * 2.0 ** -8 + 2 * rounding(layer.double(), BF))


# ------------------------------------------------------------------ all of them together

def block(sp, state):
    """What a transformer block does before its attention, for one set of rows."""
    q, scale, h = sp.spconv_rms_norm_q8(state["x"], state["weight"], residual=state["h"], sum_out=state["h2"])
    qkv = sp.spconv_linear_w4(q, *state["w4"], bias=state["bias"], x_scale=scale)
    heads = qkv[:, :2 * state["c"]].unflatten(1, (-1, 64))
    sp.spconv_rope_apply(state["rope"], state["coords"], heads, out=heads)
    y = sp.spconv_rms_norm(state["x"], state["weight"], residual=state["h"], rstd=state["rstd"])[0]
    dx, dw = sp.spconv_rms_norm_backward(state["x"], h, state["weight"], state["rstd"], dsum=y)
    return qkv, h, y, dx, dw


def block_state(sp, n, c, seed):
    packed, s, z = sp.spconv_w4_quantize((randn(c, 3 * c, seed=seed) * c ** -0.5).to(BF), 64)
    return dict(x=randn(n, c, seed=seed + 1, dtype=BF), h=randn(n, c, seed=seed + 2, dtype=BF),
                h2=torch.empty((n, c), dtype=BF, device="cuda"), weight=(1 + 0.1 * randn(c, seed=seed + 3)).to(BF),
                w4=(packed, s, z), bias=randn(3 * c, seed=seed + 4, dtype=BF), coords=coords_for(n, 64, seed),
                rope=sp.spconv_rope_create(64), rstd=torch.empty(n, device="cuda"), c=c)


@pytest.mark.parametrize("n", [1, 20, 32])
def test_block_chain(sp, n):
    c = 256
    st = block_state(sp, n, c, 0)
    qkv, h, *_ = block(sp, st)
    y, h_ref, _ = ref.rms_norm(st["x"], st["weight"], st["h"], 1e-6)
    within(h, h_ref, rounding(h_ref, BF) + U * h_ref.abs())
    # 8-bit rows: half a step of e4m3 on each element, 2^-4 of it or 2^-10 of the row's scale, through |W|
    s = y.abs().amax(1, keepdim=True) / 448
    dq = torch.maximum(y.abs() * 2.0 ** -4, s * 2.0 ** -10) * 1.001
    want, err = ref.linear_w4(y.float(), *st["w4"], st["bias"], None)
    codes = ref.w4_codes(st["w4"][0]).double()
    wmat = codes * st["w4"][1].double().repeat_interleave(64, 1) + st["w4"][2].double().repeat_interleave(64, 1)
    spread = dq @ wmat.abs().t() + err + rounding(want, BF)
    within(qkv[:, 2 * c:], want[:, 2 * c:], spread[:, 2 * c:])
    pre = want[:, :2 * c].unflatten(1, (-1, 64))
    turned, mag = ref.rope(pre, st["coords"], *ref.rope_default(64), "interleaved", False)
    sp_mag = spread[:, :2 * c].unflatten(1, (-1, 32, 2)).sum(3, keepdim=True).expand(-1, -1, -1, 2).flatten(2)
    got = qkv[:, :2 * c].unflatten(1, (-1, 64))
    within(got, turned, sp_mag + rope_tol(turned, mag + sp_mag, BF))


def test_captured_replayed_and_on_another_stream(sp):
    """The block captured twice (two graphs, other data), replayed in turn and together on
    two streams, and run eagerly on a side stream given by argument."""
    states = [block_state(sp, n, 256, 50 * n) for n in (3, 32)]
    want = [[t.clone() for t in block(sp, st)] for st in states]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for st in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(block(sp, st))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for t in outs[0] + outs[1]:
            t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))
    # new data through the captured graph
    fresh = block_state(sp, 3, 256, 999)
    states[0]["x"].copy_(fresh["x"])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], block(sp, states[0])))
    # a stream by argument: the call waits for nothing else, the caller orders the streams
    st, side = states[1], torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        q, scale, h = sp.spconv_rms_norm_q8(st["x"].t().contiguous().t(), st["weight"], residual=st["h"], stream=stream)
        lin = sp.spconv_linear_w4(q, *st["w4"], bias=st["bias"], x_scale=scale, stream=stream)
        turned = sp.spconv_rope_apply(st["rope"], st["coords"], lin[:, :512].unflatten(1, (-1, 64)), stream=stream)
        dx, dw = sp.spconv_rms_norm_backward(st["x"], h, st["weight"], st["rstd"], dsum=want[1][2], stream=stream)
        side.synchronize()
        assert torch.equal(turned.flatten(1), want[1][0][:, :512]) and torch.equal(h, want[1][1])
        assert torch.equal(dx, want[1][3]) and torch.equal(dw, want[1][4])


def test_offsets_past_32_bits(sp):
    """More than 2^31 elements: the last rows are right."""
    n, c = (1 << 21) + 5, 1024
    x = torch.zeros((n, c), dtype=BF, device="cuda")
    x[:3] = randn(3, c, seed=1, dtype=BF)
    x[-70:] = randn(70, c, seed=2, dtype=BF)
    w = (1 + 0.1 * randn(c, seed=3)).to(BF)
    rows = torch.tensor([0, 1, 2, n - 70, n - 1], device="cuda")
    out, rstd = torch.empty_like(x), torch.empty(n, device="cuda")
    sp.spconv_rms_norm(x, w, out=out, rstd=rstd)
    y, _, _ = ref.rms_norm(x[rows], w, None, 1e-6)
    within(out[rows], y, rounding(y, BF) + chain(c) * U * y.abs())
    q, s = sp.spconv_rms_norm_q8(x, w)
    check_q8(q[rows], s[rows], y, c)
    del q
    dx, dw = sp.spconv_rms_norm_backward(out, x, w, rstd, dx=None)
    alive = torch.cat([torch.arange(3), torch.arange(n - 70, n)]).cuda()
    want, wantw, mag, magw = ref.rms_norm_backward(out[alive], x[alive], w, rstd[alive], None)
    within(dx[alive], want, rounding(want, BF) + (chain(c) + 4) * U * mag)
    within(dw, wantw, (73 + 40) * U * magw)  # the other rows add exact zeros
    del dx, out
    heads = x.unflatten(1, (16, 64))
    coords = coords_for(n, 4096)
    rope = sp.spconv_rope_create(64)
    turned = sp.spconv_rope_apply(rope, coords, heads)
    want, mag = ref.rope(heads[rows], coords[rows], *ref.rope_default(64), "interleaved", False)
    within(turned[rows], want, rope_tol(want, mag, BF))


def test_binding_refusals_on_device(sp):
    x, w = randn(4, 16, dtype=BF), randn(16, dtype=BF)
    f32 = torch.zeros(4, device="cuda")
    for fn in (lambda: sp.spconv_rms_norm(x, w.float()), lambda: sp.spconv_rms_norm(x, w[:8]),
               lambda: sp.spconv_rms_norm(x, w, residual=x[:3]), lambda: sp.spconv_rms_norm(x, w, sum_out=x),
               lambda: sp.spconv_rms_norm(x, w, out=torch.empty((16, 4), dtype=BF, device="cuda").t()),
               lambda: sp.spconv_rms_norm(x, w, rstd=f32[:3]), lambda: sp.spconv_rms_norm(x.half()),
               lambda: sp.spconv_rms_norm(x, w.cpu()), lambda: sp.spconv_rms_norm_q8(x, w, out=torch.empty_like(x)),
               lambda: sp.spconv_rms_norm_backward(x, x, w, f32.double()),
               lambda: sp.spconv_rms_norm_backward(x[:2], x, w, f32)):
        with pytest.raises(ValueError):
            fn()
    for fn in (lambda: sp.spconv_rms_norm(x, w, out=x), lambda: sp.spconv_rms_norm(x, w, eps=-1.0),
               lambda: sp.spconv_rms_norm_backward(x, x, w, f32, dx=x)):
        with pytest.raises(sp.SpconvError):
            fn()
    rope = sp.spconv_rope_create(8)
    h = x.unflatten(1, (2, 8))
    c = torch.zeros((4, 4), dtype=torch.int32, device="cuda")
    for fn in (lambda: sp.spconv_rope_apply(rope, c[:3], h), lambda: sp.spconv_rope_apply(rope, c.long(), h),
               lambda: sp.spconv_rope_apply(rope, c, x), lambda: sp.spconv_rope_apply(rope, c.cpu(), h),
               lambda: sp.spconv_rope_apply(rope, c, h, out=h[:, :1])):
        with pytest.raises(ValueError):
            fn()
    with pytest.raises(sp.SpconvError):
        sp.spconv_rope_apply(rope, c[:2], h[:2], out=h[1:3])
    p, s, z = w4_inputs(64, 8, 32, BF)
    xx = randn(33, 64, dtype=BF)
    for fn in (lambda: sp.spconv_linear_w4(xx[:2].float(), p, s, z), lambda: sp.spconv_linear_w4(xx[:2, :32], p, s, z),
               lambda: sp.spconv_linear_w4(xx[:2], p, s, z[:, :1]), lambda: sp.spconv_linear_w4(xx[:2], p.long(), s, z),
               lambda: sp.spconv_linear_w4(xx[:2], p, s, z, x_scale=f32[:2]),
               lambda: sp.spconv_linear_w4(xx[:2], p, s, z, bias=s[0]), lambda: sp.spconv_w4_quantize(xx, 64)):
        with pytest.raises(ValueError):
            fn()
    with pytest.raises(sp.SpconvError) as e:
        sp.spconv_linear_w4(xx, p, s, z)
    assert e.value.status == sp.UNSUPPORTED
