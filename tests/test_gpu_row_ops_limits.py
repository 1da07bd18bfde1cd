"""The operators on feature rows (RMS norm, rotary positions, 4-bit linear layer) where a
last bit, a lost row or a far angle would show: exact results, and bounds counted from the
launches' own chains of additions."""
import math
from fractions import Fraction

import pytest
import torch

import row_ops_bounds as bounds
from row_ops_bounds import U

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sp():
    import submanifold_sparse_convolution_submconv3d_b200 as p
    return p


# ------------------------------------------------------------------ 8-bit rows

def signs(n, c, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 1.0 - 2.0 * torch.randint(0, 2, (n, c), generator=g, device="cuda").float()


def next_to_middles(c, scale):
    """fp32 weights up to 448 scale, the others up to 3 last bits around scale times the
    middles between neighbouring e4m3 values, normal ones and those under 2^-6."""
    i = torch.arange(c, device="cuda")
    codes = i * 11 % 125
    values = torch.arange(126, device="cuda").to(torch.uint8).view(torch.float8_e4m3fn).float()
    middle = 0.5 * (values[codes] + values[codes + 1])
    bits = (middle * scale).view(torch.int32) + (i // 125 % 7 - 3).to(torch.int32)
    w = bits.view(torch.float32).clone()
    w[c // 2] = 448.0 * scale
    return w


def same(a, b):
    """Bit for bit as far as values go: any NaN equals any NaN."""
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(nan=0.0), b.nan_to_num(nan=0.0))


def check_codes(sp, n, c, w):
    """Rows of +-1 have a sum of squares of exactly c, so 1 / rms is the same number in
    every launch, and the fp32 norm of the same rows is the y that the codes are made of."""
    x = signs(n, c, seed=c)
    y = sp.spconv_rms_norm(x, w.float(), eps=0.0)
    scale = y.abs().amax(1)
    scale = (scale / torch.full_like(scale, 448.0)).clamp(min=2.0 ** -126)  # (by a number torch multiplies by 1 / 448)
    want = (y / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    q, s = sp.spconv_rms_norm_q8(x.to(w.dtype), w, eps=0.0)
    assert same(s, scale)
    assert same(q.float(), want)


@pytest.mark.parametrize("n,c", [(5, 16), (5, 24), (9, 48), (70, 64), (70, 80), (70, 128), (33, 160), (33, 250), (20, 333),
                                 (20, 384), (20, 500), (9, 640), (9, 1001), (9, 1024), (2400, 1408), (9, 1408), (5, 2048),
                                 (5, 4000), (3, 5518), (3, 8192), (2, 16000), (2, 32768), (2, 40001)])
def test_q8_codes_are_the_rounded_quotients(sp, n, c):
    for scale in (0.7123, 1.9999, 3.0e-5, 7.7e20):
        check_codes(sp, n, c, next_to_middles(c, scale))
    # bf16: scales p 2^k whose reciprocals are rounded, weights on the middles themselves
    for p in (3.0, 5.0, 7.0):
        w = next_to_middles(c, p / 64)
        check_codes(sp, n, c, w.to(BF))


@pytest.mark.parametrize("c", [16, 80, 128, 333, 1024, 5518, 40001])
def test_q8_codes_of_extreme_scales(sp, c):
    """The smallest scale (2^-126, its reciprocal exact), the largest, an infinite one and NaN."""
    for dtype in (F32, BF):
        w = torch.full((c,), 2.0 ** -130, device="cuda", dtype=dtype)
        w[::3] = 0
        check_codes(sp, 4, c, w)
        w = torch.full((c,), 1.5 * 2.0 ** 126, device="cuda", dtype=dtype)
        w[1::2] = 2.0 ** 117
        check_codes(sp, 4, c, w)
        w[c // 3] = float("inf")     # its own code NaN, the finite ones 0
        check_codes(sp, 4, c, w)
        w[c // 3] = float("nan")
        check_codes(sp, 4, c, w)


# ------------------------------------------------------------------ far angles

PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679821, 10 ** 103)


def exact_turns(freqs, coords):
    """cos and sin of freqs[j] * coords[i] in 64 bits, the turn reduced in whole numbers."""
    t = [[float((Fraction(f) * c / (2 * PI) + Fraction(1, 2)) % 1 - Fraction(1, 2)) for f in freqs] for c in coords]
    t = torch.tensor(t, dtype=torch.float64, device="cuda") * (2 * math.pi)
    return t.cos(), t.sin()


def turned_units(sp, freqs, coords, dtype):
    """What a pair (1, 0) becomes: (cos, sin) of every voxel and frequency."""
    rope = sp.spconv_rope_create(2 * len(freqs), freqs=freqs, axes=[1] * len(freqs))
    at = torch.zeros((len(coords), 4), dtype=torch.int32, device="cuda")
    at[:, 2] = torch.tensor(coords, dtype=torch.int32)
    x = torch.tensor([1.0, 0.0], device="cuda", dtype=dtype).repeat(len(freqs)).expand(len(coords), 1, -1).contiguous()
    out = sp.spconv_rope_apply(rope, at, x)[:, 0]
    return out[:, 0::2].double(), out[:, 1::2].double()


FAR = [0, 1, -1, 7, 1000, -65535, 123456789, 2 ** 31 - 1, -2 ** 31]


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rope_turns_of_any_frequency(sp, dtype):
    """The fraction of a turn keeps its bits however large the frequency is.  Bound: the
    cosine and sine of the rounded angle (2^-21 of the pair; bf16 2^-20) and the result's rounding."""
    freqs = [1.0, 40.0, -40.0, 1e3, 65536.5, 1e9, -1e12, 3e15, 2.0 ** 53 + 2, 1e19, -1.8e19, 2 * math.pi, 1e-9, 2.0 ** -60]
    freqs += [0.3 * 10.0 ** k for k in range(-4, 14)]
    tol = (2.0 ** -20 if dtype == BF else 2.0 ** -21) + torch.finfo(dtype).eps / 2
    for got, want in zip(turned_units(sp, freqs, FAR, dtype), exact_turns(freqs, FAR)):
        assert float((got - want).abs().max()) <= tol


def test_rope_fp32_angles_are_near_to_the_last_bit(sp):
    """Angles within 2^-32 of a turn, also where the sine nearly vanishes: 1.5 2^-33 of a turn
    (2^-34 of the frequency's fraction at coordinate 2^31, 2^-33 of the product's rounding) is
    under 2^-29 rad; the sine and cosine themselves 2 last bits (2^-22), one operation 2^-24."""
    freqs = [math.pi * k * (1 + 2.0 ** -m) for m in range(10, 30) for k in (0.25, 0.5, 1.0, 2.0)]
    freqs += [0.7 ** k for k in range(30)] + [-0.37, 40.0, 1e6]
    for got, want in zip(turned_units(sp, freqs, FAR, F32), exact_turns(freqs, FAR)):
        assert ((got - want).abs() <= want.abs() * (2.0 ** -22 + 2.0 ** -24) + 2.0 ** -29).all()


# ------------------------------------------------------------------ sums of the norm and its gradient

def within(got, want, tol, what=""):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist())


def randn(*shape, seed=0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,c", [(70, 8), (70, 16), (70, 31), (70, 64), (70, 96), (70, 128), (33, 190), (33, 256), (33, 384),
                                 (20, 512), (20, 513), (9, 768), (9, 1024), (2400, 1408), (9, 2048), (5, 2049), (5, 4096),
                                 (3, 8192), (3, 16383), (2, 32768), (2, 32769), (1, 65536)])
def test_rms_norm_within_its_own_chain(sp, n, c, dtype):
    x, r, w = randn(n, c, seed=c, dtype=dtype) * 2, randn(n, c, seed=1, dtype=dtype), (1 + 0.3 * randn(c, seed=2)).to(dtype)
    rstd = torch.empty(n, device="cuda")
    out, _ = sp.spconv_rms_norm(x, w, residual=r, eps=1e-6, rstd=rstd)
    h = x.double() + r.double()
    want = 1.0 / torch.sqrt((h * h).mean(1) + 1e-6)
    y = h * want[:, None] * w.double()
    half = torch.finfo(dtype).eps / 2
    within(rstd, want, bounds.rstd_bound(c) * want, "rstd")
    # (the result's rounding, and that of values that only rounding carries over)
    within(out, y, y.abs() * (half + bounds.norm_bound(c) * (1 + half)), "out")
    q, s = sp.spconv_rms_norm_q8(x, w, residual=r, eps=1e-6)[:2]
    top = y.abs().amax(1) / 448
    within(s, top, (bounds.norm_bound(c) + U) * top, "scale")
    v = q.double() * s.double()[:, None]
    within(v, y, torch.maximum(y.abs() * 2.0 ** -4, top[:, None] * 2.0 ** -10) * (1 + 2 * bounds.norm_bound(c)) + y.abs() * 2 * bounds.norm_bound(c), "q")


GRADIENTS = [  # one CTA alone, several turns of one, a few CTAs, several turns of all; every count of threads a row
    (1, 16), (40, 16), (1000, 16), (1025, 16), (2051, 24), (40001, 9), (120000, 32), (70001, 33), (50001, 64), (30001, 120),
    (17, 256), (40000, 250), (9001, 256), (129, 512), (16, 513), (17, 513), (7001, 500), (5001, 512), (3001, 1024), (5, 2048),
    (2001, 2047), (1501, 4096), (4, 4096), (901, 4104), (701, 8192), (701, 8191), (303, 12000), (3, 16384), (451, 9001),
    (300, 16390), (4, 20000), (299, 20001), (700, 33000), (2, 65536)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,c", GRADIENTS)
def test_rms_norm_weight_gradient_loses_no_row(sp, n, c, dtype):
    """Whole numbers under 2^24 in all sums: exact in any order, so one lost or doubled row shows."""
    g = torch.Generator(device="cuda").manual_seed(n + c)
    most = 8 if n * 64 < 1 << 24 else 6
    dy = torch.randint(1, most + 1, (n, c), generator=g, device="cuda").to(dtype)
    h = torch.randint(1, most + 1, (n, c), generator=g, device="cuda").to(dtype)
    w = torch.randint(1, 4, (c,), generator=g, device="cuda").to(dtype)
    want = (dy.double() * h.double()).sum(0)
    assert float(want.max()) < 2 ** 24
    for dsum in (None, dy):
        dx, dw = sp.spconv_rms_norm_backward(dy, h, w, torch.ones(n, device="cuda"), dsum=dsum)
        assert torch.equal(dw.double(), want)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,c", GRADIENTS)
def test_rms_norm_gradient_within_its_own_chains(sp, n, c, dtype):
    h, dy, d = (randn(n, c, seed=c + k, dtype=dtype) for k in range(3))
    w = (1 + 0.3 * randn(c, seed=3)).to(dtype)
    rstd = (1 + 0.2 * randn(n, seed=4)).abs() + 0.1
    hd, dyd, rd = h.double(), dy.double(), rstd.double()[:, None]
    xh, g = hd * rd, dyd * w.double()
    mean, meanm = (g * xh).mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    half = torch.finfo(dtype).eps / 2
    for dsum in (None, d):
        dx, dw = sp.spconv_rms_norm_backward(dy, h, w, rstd, dsum=dsum)
        want, mag = rd * (g - xh * mean), rd * (g.abs() + xh.abs() * meanm)
        if dsum is not None:
            want, mag = want + dsum.double(), mag + dsum.double().abs()
        within(dx, want, want.abs() * half + (1 + half) * bounds.dx_bound(c) * mag, "dx")
        item, per_thread = (4, 8) if dtype == F32 else (8, 16)
        within(dw, (dyd * xh).sum(0), bounds.column_bound(n, c, item, per_thread) * (dyd * xh).abs().sum(0), "dweight")
