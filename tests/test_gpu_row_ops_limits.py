"""The operators on feature rows (RMS norm, rotary positions, 4-bit linear layer) where a
last bit, a lost row or a far angle would show: exact results, and bounds counted from the
launches' own chains of additions."""
import pytest
import torch

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
