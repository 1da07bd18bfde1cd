"""Cases for measuring the feature-row operators: RMS norm with the residual's
addition (forward, 8-bit output, backward), rotary positions from voxel
coordinates, and the linear layer with 4-bit weights.

``run`` computes them in elementary torch operations in 32 bits, or, where ``own``
is true, through the package's entry points; ``exact`` computes them in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_EPS = 1e-6
_E4M3_MAX = 448.0
_MIN_SCALE = 2.0 ** -126


def listed():
    return [
        # one token (or one modulation vector) of a 1024-channel block: latency alone
        {"name": "norm_one_row", "op": "norm", "n": 1, "c": 1024, "dtype": "bf16", "residual": True, "train": False},
        # the residual stream of the four 64^3 shell shapes, 512 channels, with what training keeps
        {"name": "norm_batched512", "op": "norm", "n": 61463, "c": 512, "dtype": "bf16", "residual": True, "train": True},
        # an odd channel count in fp32, as a head with a few extra channels has it: rows off the 16-byte grid
        {"name": "norm_odd_f32", "op": "norm", "n": 20011, "c": 333, "dtype": "f32", "residual": False, "train": True},
        # the stream of a wide block on the 64^3 shapes, written as 8-bit rows for an 8-bit layer
        {"name": "norm_q8_wide", "op": "norm_q8", "n": 61463, "c": 1024, "dtype": "bf16", "residual": True},
        # training on the uniform 128^3 set, 128 channels: many short rows, one long column sum
        {"name": "norm_bwd_uniform128", "op": "norm_bwd", "n": 209715, "c": 128, "dtype": "bf16", "residual": True},
        # training of a wide block on a latent set: few long rows
        {"name": "norm_bwd_wide", "op": "norm_bwd", "n": 8191, "c": 4096, "dtype": "bf16", "residual": False},
        # the queries of one new token
        {"name": "rope_one_row", "op": "rope", "n": 1, "heads": 16, "d": 64, "dtype": "bf16", "layout": "interleaved",
         "inverse": False, "packed": False, "extent": 64},
        # queries or keys of the 256^3 shells, read out of the packed projection [n, 3, heads, d]
        {"name": "rope_shells256", "op": "rope", "n": 273995, "heads": 12, "d": 64, "dtype": "bf16",
         "layout": "interleaved", "inverse": False, "packed": True, "extent": 256},
        # the gradient, fp32, halves layout, far positions
        {"name": "rope_grad_far", "op": "rope", "n": 16934, "heads": 8, "d": 96, "dtype": "f32", "layout": "halves",
         "inverse": True, "packed": False, "extent": 65535},
        # one token through a square block matrix
        {"name": "w4_one_row", "op": "w4", "n": 1, "cin": 4096, "cout": 4096, "group": 64, "dtype": "bf16",
         "x8": False, "bias": True},
        # a few 8-bit rows through a large matrix
        {"name": "w4_rows8_x8", "op": "w4", "n": 8, "cin": 8192, "cout": 16384, "group": 128, "dtype": "bf16",
         "x8": True, "bias": False},
        # a small latent set, fp32, odd output count, short groups
        {"name": "w4_rows27_f32", "op": "w4", "n": 27, "cin": 1504, "cout": 2051, "group": 32, "dtype": "f32",
         "x8": False, "bias": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_q8", "norm_bwd", "rope", "w4"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_q8", "norm_bwd"):
        c = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            c = (c + 15) // 16 * 16
        n = _log(rng, 1, max(2, min(300000, 24000000 // c)))
        case = {"op": op, "n": n, "c": c, "dtype": dtype, "residual": rng.random() < 0.5}
        if op == "norm":
            case["train"] = rng.random() < 0.5
        return case
    if op == "rope":
        d = rng.choice([32, 48, 64, 80, 96, 128, 256])
        heads = rng.randint(1, 32)
        n = _log(rng, 1, max(2, min(270000, 50000000 // (heads * d))))
        return {"op": op, "n": n, "heads": heads, "d": d, "dtype": dtype, "layout": rng.choice(["interleaved", "halves"]),
                "inverse": rng.random() < 0.5, "packed": rng.random() < 0.5, "extent": _log(rng, 8, 65535)}
    group = rng.choice([32, 64, 128])
    cin = max(group, _log(rng, 128, 8192) // group * group)
    cout = _log(rng, 64, 16384)
    n = min(rng.choice([1, 1, 2, 3, 4, 7, 8, 12, 16, 24, 32]), max(1, (1 << 30) // (cin * cout)))
    x8 = dtype == "bf16" and rng.random() < 0.4
    return {"op": op, "n": n, "cin": cin, "cout": cout, "group": group, "dtype": dtype, "x8": x8,
            "bias": rng.random() < 0.5}


def _rope_table(d, base=10000.0):
    """(frequency, axis) of each pair: d // 6 pairs an axis, one ladder base^(-j / P)
    per axis in the order x, y, z; the pairs left over do not turn (axis -1)."""
    per = d // 2 // 3
    ladder = torch.pow(torch.tensor(base, dtype=torch.float64), -torch.arange(per, dtype=torch.float64) / max(per, 1))
    rest = d // 2 - 3 * per
    freqs = torch.cat([ladder, ladder, ladder, torch.zeros(rest, dtype=torch.float64)])
    axes = torch.cat([torch.full((per,), a) for a in (0, 1, 2)] + [torch.full((rest,), -1)])
    return freqs, axes


def _inputs(case, seed):
    """The inputs of a case, on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    dt = _DTYPES[case["dtype"]]
    op, n = case["op"], case["n"]
    s = {"case": case}
    if op in ("norm", "norm_q8", "norm_bwd"):
        c = case["c"]
        # a residual stream: unit rows of differing size, a few channels far above the others
        channel = torch.exp(0.5 * normal(c))
        row = torch.exp(0.5 * normal(n, 1))
        s["x"] = (normal(n, c).mul_(channel).mul_(row)).to(dt)
        s["weight"] = (1.0 + 0.2 * normal(c)).to(dt)
        s["residual"] = (normal(n, c).mul_(channel)).to(dt) if case["residual"] else None
        if op == "norm_bwd":
            s["dy"] = normal(n, c).to(dt)
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + _EPS)
    elif op == "rope":
        heads, d = case["heads"], case["d"]
        if case["packed"]:
            s["x"] = normal(n, 3, heads, d).to(dt)[:, 1]
        else:
            s["x"] = normal(n, heads, d).to(dt)
        s["coords"] = torch.randint(0, case["extent"], (n, 4), generator=g, device="cuda", dtype=torch.int32)
        s["coords"][:, 0] = 0
        freqs, axes = _rope_table(d)
        s["freqs"], s["axes"] = freqs.cuda(), axes.cuda()
    else:
        cin, cout, group = case["cin"], case["cout"], case["group"]
        s["packed"] = torch.randint(-2 ** 31, 2 ** 31, (cout, cin // 8), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        scale = (0.5 + torch.rand((cout, cin // group), generator=g, device="cuda")) * (0.25 * cin ** -0.5)
        s["scales"] = scale.to(dt)
        s["offsets"] = (scale * (-7.5 + 0.5 * normal(cout, cin // group))).to(dt)
        s["bias"] = normal(cout).mul_(0.1).to(dt) if case["bias"] else None
        x = normal(n, cin)
        if case["x8"]:
            s["x_scale"] = x.abs().amax(1) / _E4M3_MAX
            s["x"] = (x / s["x_scale"][:, None]).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn)
        else:
            s["x"], s["x_scale"] = x.to(dt), None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import submanifold_sparse_convolution_submconv3d_b200 as sp
        s["sp"] = sp
        if case["op"] == "rope":
            s["rope"] = sp.spconv_rope_create(case["d"], layout=case["layout"])
    return s


def _run_own(s):
    sp, case = s["sp"], s["case"]
    op = case["op"]
    if op == "norm":
        rstd = torch.empty(case["n"], dtype=torch.float32, device="cuda") if case["train"] else None
        out = sp.spconv_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=_EPS, rstd=rstd)
        return (out if s["residual"] is not None else (out,)) + ((rstd,) if case["train"] else ())
    if op == "norm_q8":
        return sp.spconv_rms_norm_q8(s["x"], s["weight"], residual=s["residual"], eps=_EPS)
    if op == "norm_bwd":
        return sp.spconv_rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], dsum=s["residual"])
    if op == "rope":
        return sp.spconv_rope_apply(s["rope"], s["coords"], s["x"], inverse=case["inverse"])
    return sp.spconv_linear_w4(s["x"], s["packed"], s["scales"], s["offsets"], bias=s["bias"], x_scale=s["x_scale"])


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], _DTYPES[case["dtype"]]
    if op in ("norm", "norm_q8"):
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        rstd = torch.rsqrt((h * h).mean(1) + _EPS)
        y = h * rstd[:, None] * s["weight"].float()
        if op == "norm":
            out = (y.to(dt),)
        else:
            scale = (y.abs().amax(1) / _E4M3_MAX).clamp(min=_MIN_SCALE)
            out = ((y / scale[:, None]).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn), scale)
        if s["residual"] is not None:
            out += (h.to(dt),)
        return out + ((rstd,) if case.get("train") else ())
    if op == "norm_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = s["x"].float() * rstd
        g = dy * s["weight"].float()
        dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
        if s["residual"] is not None:
            dx = dx + s["residual"].float()
        return dx.to(dt), (dy * xh).sum(0)
    if op == "rope":
        x = s["x"].float()
        # far positions need the angle in 64 bits
        pos = s["coords"][:, 1:].double()[:, s["axes"].clamp(min=0)]
        angle = pos * s["freqs"]
        if case["inverse"]:
            angle = -angle
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        half = case["d"] // 2
        if case["layout"] == "interleaved":
            a, b = x[..., 0::2], x[..., 1::2]
            return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(2).to(dt)
        a, b = x[..., :half], x[..., half:]
        return torch.cat((a * cos - b * sin, a * sin + b * cos), -1).to(dt)
    shifts = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    q = ((s["packed"][:, :, None] >> shifts) & 15).float().view(case["cout"], -1, case["group"])
    w = (q * s["scales"].float()[:, :, None] + s["offsets"].float()[:, :, None]).view(case["cout"], -1)
    out = s["x"].float() @ w.t()
    if s["x_scale"] is not None:
        out = out * s["x_scale"][:, None]
    if s["bias"] is not None:
        out = out + s["bias"].float()
    return out.to(dt)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def exact(case, seed):
    """The definition in 64 bits, unrounded: the outputs of ``run`` in the same order."""
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("norm", "norm_q8"):
        h = s["x"].double()
        if s["residual"] is not None:
            h += s["residual"].double()
        norm = torch.sqrt(torch.einsum("nc,nc->n", h, h) / case["c"] + _EPS)
        y = torch.einsum("nc,c,n->nc", h, s["weight"].double(), 1.0 / norm)
        if op == "norm":
            out = [y]
        else:
            scale = torch.maximum(torch.linalg.vector_norm(y, float("inf"), dim=1) / _E4M3_MAX,
                                  torch.full_like(norm, _MIN_SCALE))
            out = [y / scale[:, None], scale]
        if s["residual"] is not None:
            out.append(h)
        if case.get("train"):
            out.append(1.0 / norm)
        return tuple(out)
    if op == "norm_bwd":
        # the rows' Jacobian w rstd (I - x x^T rstd^2 / c), applied from the left
        x, dy, r = s["x"].double(), s["dy"].double(), s["rstd"].double()
        wdy = dy * s["weight"].double()
        along = torch.einsum("nc,nc->n", wdy, x) * r.pow(3) / case["c"]
        dx = torch.einsum("nc,n->nc", wdy, r) - torch.einsum("nc,n->nc", x, along)
        if s["residual"] is not None:
            dx += s["residual"].double()
        return dx, torch.einsum("nc,nc,n->c", dy, x, r)
    if op == "rope":
        # complex rotation of each pair
        x, n, heads, half = s["x"].double(), case["n"], case["heads"], case["d"] // 2
        inter = case["layout"] == "interleaved"
        pairs = x.reshape(n, heads, half, 2) if inter else x.reshape(n, heads, 2, half).transpose(2, 3)
        z = torch.view_as_complex(pairs.contiguous())
        three = torch.zeros((3, half), dtype=torch.float64, device="cuda")
        turning = s["axes"] >= 0
        three[s["axes"][turning], torch.arange(half, device="cuda")[turning]] = s["freqs"][turning]
        angle = s["coords"][:, 1:].double() @ three
        turn = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)
        out = torch.view_as_real(z * turn[:, None])
        return (out if inter else out.transpose(2, 3)).reshape(n, heads, 2 * half)
    cin, cout, group = case["cin"], case["cout"], case["group"]
    words = s["packed"].to(torch.int64) & 0xFFFFFFFF
    q = torch.stack([(words // 16 ** i) % 16 for i in range(8)], -1).reshape(cout, cin // group, group).double()
    x = s["x"].double().reshape(case["n"], cin // group, group)
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double()[:, None, None]
    out = torch.einsum("ngk,ogk,og->no", x, q, s["scales"].double()) \
        + torch.einsum("ng,og->no", x.sum(2), s["offsets"].double())
    if s["bias"] is not None:
        out = out + s["bias"].double()
    return out


def work(case):
    op, n, e = case["op"], case["n"], _BYTES[case["dtype"]]
    if op in ("norm", "norm_q8"):
        c, r = case["c"], 2 if case["residual"] else 0  # the residual in, the sum out
        out = n * c * e if op == "norm" else n * (c + 4)
        return {"bytes": n * c * e * (1 + r) + out + c * e + (4 * n if case.get("train") else 0), "flops": 6 * n * c}
    if op == "norm_bwd":
        c = case["c"]
        return {"bytes": n * c * e * (4 if case["residual"] else 3) + c * (e + 4) + 4 * n, "flops": 10 * n * c}
    if op == "rope":
        elems = n * case["heads"] * case["d"]
        return {"bytes": 2 * elems * e + 16 * n, "flops": 3 * elems}
    cin, cout, x = case["cin"], case["cout"], 1 if case["x8"] else e
    return {"bytes": cout * cin // 2 + 2 * e * cout * (cin // case["group"]) + n * cin * x + n * cout * e
            + (4 * n if case["x8"] else 0) + (cout * e if case["bias"] else 0), "flops": 2 * n * cin * cout}
