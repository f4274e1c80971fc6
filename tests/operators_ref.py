"""Definitions in 64 bits of the operators around the FP8 GEMMs (norm, gated
activation, ragged products), for the tests; no code shared with the kernels.

Bounds.  u = 2^-24 is half an fp32 ulp.  A bf16 output may be off by its
rounding (2^-8 of its value at most), an e4m3 code by half its spacing, and
either by what the fp32 arithmetic before it loses.
"""
import torch

F64 = torch.float64
FLOOR = 1e-4
U32 = 2.0 ** -24
BF16_ROUND = 2.0 ** -8


def groups(y):
    return y.unflatten(-1, (-1, 128))


def group_amax(y):
    return groups(y).abs().amax(-1).clamp_min(FLOOR)


def norm(x, r, w, eps):
    h = x.to(F64) + (r.to(F64) if r is not None else 0.0)
    rstd = 1.0 / torch.sqrt((h * h).mean(-1) + eps)
    return h, rstd, h * rstd[:, None] * w.to(F64)


def norm_backward(dy, h, rstd, w, dr):
    dy, h, rstd, w = dy.to(F64), h.to(F64), rstd.to(F64), w.to(F64)
    xh = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - xh * (g * xh).mean(-1, keepdim=True))
    if dr is not None:
        dx = dx + dr.to(F64)
    return dx, (dy * xh).sum(0)


def swiglu(gu):
    g, u = gu.to(F64).chunk(2, dim=-1)
    return g * torch.sigmoid(g) * u


def swiglu_backward(gu, dy):
    g, u = gu.to(F64).chunk(2, dim=-1)
    dy, s = dy.to(F64), torch.sigmoid(g)
    return torch.cat([dy * u * s * (1.0 + g * (1.0 - s)), dy * g * s], -1)


def products(form, a, b, sizes, c=None, rows=None):
    """(D, S): the product and the same sum over magnitudes (for the bounds)."""
    a, b = a.to(F64), b.to(F64)
    out, mag, first = [], [], 0
    for e, n in enumerate(sizes):
        x = a[first:first + n]
        if form == "tn":
            y = b[first:first + n]
            out.append(x.t() @ y)
            mag.append(x.t().abs() @ y.abs())
        else:
            w = b[e].t() if form == "nt" else b[e]
            out.append(x @ w)
            mag.append(x.abs() @ w.abs())
        first += n
    d, s = (torch.stack(out), torch.stack(mag)) if form == "tn" else (torch.cat(out), torch.cat(mag))
    if c is not None:
        d, s = d + c.to(F64), s + c.to(F64).abs()
    return d, s


def scales(sa, M, kb):
    """K-group-major fp32 scales [..., kb, ld] -> [..., M, kb]."""
    return sa[..., :kb, :M].transpose(-1, -2)


def unpack_ue8m0(words, M, kb):
    """Packed words int32 [..., ceil(kb/4), ld] -> scales in 64 bits [..., M, kb]."""
    b = words.contiguous().view(torch.uint8).unflatten(-1, (-1, 4))     # [..., kbp, ld, 4]
    e = b.transpose(-1, -2).flatten(-3, -2)                            # [..., kbp * 4, ld]
    return torch.exp2(e[..., :kb, :M].transpose(-1, -2).to(F64) - 127.0)


def check_close(got, want, slack, what):
    """|got - want| <= BF16_ROUND |want| (1 + 2^-8) + slack, element by element."""
    got = got.to(F64)
    lim = BF16_ROUND * (1 + 2.0 ** -8) * want.abs() + slack
    bad = ~((got - want).abs() <= lim)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[:4].tolist()}"


def check_codes(codes, scale, y, rel, what):
    """The codes are y / scale rounded to e4m3, y known to `rel` (relative)."""
    q = codes.view(torch.float8_e4m3fn).to(F64)
    assert torch.isfinite(q).all(), f"{what}: NaN codes"
    v = groups(y) / scale[..., None]
    v = v.flatten(-2)
    # e4m3 spacing at |v|: 2^(e - 3) for 2^e <= |v| < 2^(e + 1), 2^-9 below 2^-6
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    lim = 0.5 * torch.exp2(e - 3) + rel * v.abs()
    bad = ~((q - v).abs() <= lim * (1 + 1e-9))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} codes off"


def check_scales(scale, y, rel, ue8m0, what):
    """Scales against amax / 448 (fp32), or the power of two not below it."""
    t = group_amax(y) / 448.0
    if ue8m0:
        up = torch.exp2(torch.ceil(torch.log2(t)))
        near = torch.exp2(torch.ceil(torch.log2(t * (1 + rel)))), torch.exp2(torch.ceil(torch.log2(t * (1 - rel))))
        bad = (scale != up) & (scale != near[0]) & (scale != near[1])
    else:
        bad = ~((scale.to(F64) - t).abs() <= rel * t)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} scales off"
