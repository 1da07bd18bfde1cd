"""Plain 64-bit forms of the operators on feature rows, written from their definitions,
and the error bounds their tests use.

u = 2^-24 is the rounding of one fp32 operation.  A sum of m fp32 terms whose longest
chain of additions has k steps is off by at most k u times the sum of the terms'
magnitudes.  The result's own rounding to type t adds at most finfo(t).eps / 2 of the
value; values under the type's smallest normal add its smallest step.
"""
import torch

U = 2.0 ** -24
E4M3_MAX = 448.0


def rounding(ref: torch.Tensor, dtype) -> torch.Tensor:
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) + f.smallest_normal * f.eps


def chain(c: int) -> int:
    """Additions on the longest path of a row's sum: a row is shared by at least a warp
    (c / 32 each) and joined by a tree, plus the few operations around it."""
    return c // 32 + 32


def rms_norm(x, weight, residual, eps):
    h = x.double() + (0 if residual is None else residual.double())
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None] * (1.0 if weight is None else weight.double())
    return y, h, rstd


def rms_norm_backward(dy, h, weight, rstd, dsum):
    """(dx, dweight, magnitude of dx's terms, of dweight's)."""
    dy, h, rstd = dy.double(), h.double(), rstd.double()[:, None]
    xh = h * rstd
    g = dy * (1.0 if weight is None else weight.double())
    dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    mag = rstd * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.double()
        mag = mag + dsum.double().abs()
    return dx, (dy * xh).sum(0), mag, (dy * xh).abs().sum(0)


def rope_default(d, base=10000.0):
    per = d // 2 // 3
    freqs = [base ** (-(j % per) / per) for j in range(3 * per)] + [0.0] * (d // 2 - 3 * per)
    return freqs, [j // per for j in range(3 * per)] + [-1] * (d // 2 - 3 * per)


def rope(x, coords, freqs, axes, layout, inverse):
    """(turned x, |a| + |b| of each element's pair)."""
    x = x.double()
    pos = torch.cat([coords[:, 1:], torch.zeros_like(coords[:, :1])], 1).double()[:, list(axes)]  # axis -1: 0
    t = pos * torch.tensor(freqs, dtype=torch.float64, device=x.device)
    t = (-t if inverse else t)[:, None]
    half = x.shape[2] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if layout == "interleaved" else (x[..., :half], x[..., half:])
    u, v, m = a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos(), a.abs() + b.abs()
    if layout == "interleaved":
        return torch.stack((u, v), -1).flatten(2), torch.stack((m, m), -1).flatten(2)
    return torch.cat((u, v), -1), torch.cat((m, m), -1)


def w4_codes(packed):
    words = packed.to(torch.int64) & 0xFFFFFFFF
    return torch.stack([(words >> (4 * e)) & 15 for e in range(8)], -1).flatten(1)


def linear_w4(x, packed, scales, offsets, bias, x_scale):
    """(out, bound on the fp32 error before the last rounding).

    The sums over all groups are of the size of |s| |q - 8| + |z + 8 s| + |z|, times |x|;
    their additions form chains of at most cin / 16 + 32 steps, counted at 2 u since a
    tensor core may cut instead of round.  Rows of bf16 meet 128 + q within a group, which
    the offset takes off again: at most 8 steps and 4 operations around them, at 2 u of
    |s| (q + 128) + |128 s|, times |x|, each group."""
    q = w4_codes(packed).double()
    group = q.shape[1] // scales.shape[1]
    s, z = (t.double().repeat_interleave(group, 1) for t in (scales, offsets))
    xs = x.double() * (1.0 if x_scale is None else x_scale.double()[:, None])
    out = xs @ (s * q + z).t()
    mag = xs.abs() @ (s.abs() * (q - 8).abs() + (z + 8 * s).abs() + z.abs()).t()
    if bias is not None:
        out = out + bias.double()
        mag = mag + bias.double().abs()
    err = mag * ((q.shape[1] // 16 + 32) * 2 * U)
    if x.dtype == torch.bfloat16:
        err = err + xs.abs() @ (s.abs() * (q + 256)).t() * (12 * 2 * U)
    return out, err


def w4_quantize(w, group):
    """Codes, scales and offsets of w [cin, cout] as the header defines them; the scale
    is (max - min) / 15 in fp32, rounded to w's type."""
    g = w.float().t().reshape(w.shape[1], -1, group)
    lo, hi = g.amin(2), g.amax(2)
    scales, offsets = ((hi - lo) / 15).to(w.dtype), lo.to(w.dtype)
    return g.double(), scales, offsets
