"""Plain forms in 64 bits of what stands around attention over a cache: norm and
rotation with their gradients, rows in 8 bits and their pooled keys, with bounds
that count roundings (attention itself: attn_ref.py).

u is half a step of the element type relative to the value, e32 that of 32
bits.  A norm's factor r is a sum of d squares in 32 bits under a root: off by
(d + 16) / 2 e32 of itself, the 16 for the mean, the root and eps.  An angle is
a fraction of a turn rounded to 32 bits, 2 pi 2^-26, taken from 64 bits where
position times frequency is off by 3 2^-53 of itself; sine and cosine are off by
two more steps of 2^-24: 2^-22 in all, and 2 pi 3 2^-53 of the turns."""
import math

import torch

import attn_ref as A

PAGE = 64
E32 = 2.0 ** -24


def live(b, n, lens, starts):
    """[b, n] tokens that count."""
    pos = torch.tensor(starts, dtype=torch.int64)[:, None] + torch.arange(n)
    if lens is None:
        return pos, torch.ones((b, n), dtype=torch.bool)
    return pos, (pos >= 0) & (pos < torch.tensor(lens, dtype=torch.int64)[:, None])


def angles(freqs, axis, place):
    """place [axes, b, n] -> angle [b, n, 1, pairs] and how far its sine and cosine may be off."""
    f = torch.tensor(freqs, dtype=torch.float64)
    a = place[torch.tensor(axis, dtype=torch.int64)].permute(1, 2, 0).double() * f
    off = 2.0 ** -22 + 3 * 2.0 ** -53 * a.abs()
    return a[:, :, None], off[:, :, None]


def turn(x, cos, sin, interleaved):
    n = cos.shape[-1]
    if interleaved:
        u, v = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack((u * cos - v * sin, u * sin + v * cos), -1).flatten(-2)
    else:
        u, v = x[..., :n], x[..., n:2 * n]
        y = torch.cat((u * cos - v * sin, u * sin + v * cos), -1)
    return torch.cat((y, x[..., 2 * n:]), -1)


def reach(x, off, interleaved):
    """|x_u| + |x_v| of each channel's pair times `off`; zero behind the pairs."""
    n = off.shape[-1]
    x = x.abs()
    if interleaved:
        s = ((x[..., 0:2 * n:2] + x[..., 1:2 * n:2]) * off).repeat_interleave(2, -1)
    else:
        s = ((x[..., :n] + x[..., n:2 * n]) * off).repeat(1, 1, 1, 2)
    return torch.cat((s, torch.zeros_like(x[..., 2 * n:])), -1)


def rope(x, w, angle, off, interleaved, eps, dtype, grad=None, alive=None):
    """{"o": (value, bound)} and with grad "dx" and "dw"; x [b, n, h, d] in 64 bits, alive [b, n]."""
    u = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * u
    d = x.shape[-1]
    er = (d + 16) / 2 * E32
    r = torch.ones_like(x[..., :1]) if w is None else 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    ww = torch.ones(d, dtype=torch.float64) if w is None else w
    cos, sin = torch.cos(angle), torch.sin(angle)
    y = x * r * ww
    ey = 0.0 if w is None else er + 2 * E32
    o = turn(y, cos, sin, interleaved)
    bo = reach(y, off + ey + 3 * E32, interleaved) + ey * y.abs()
    out = {"o": (o, u * (o.abs() + bo) + bo + tiny)}
    if grad is None:
        return out
    if alive is not None:
        grad = torch.where(alive[..., None, None], grad, 0.0)
        x = torch.where(alive[..., None, None], x, 0.0)
        r = torch.where(alive[..., None, None], r, 0.0)
    dy = turn(grad, cos, -sin, interleaved)
    edy = reach(grad, off + 3 * E32, interleaved)
    if w is None:
        out["dx"] = (dy, u * (dy.abs() + edy) + edy + tiny)
        return out
    rows = x.shape[0] * x.shape[1] * x.shape[2]
    out["dw"] = ((dy * x * r).sum((0, 1, 2)),
                 (edy * (x * r).abs() + (er + (rows + 4) * E32) * (dy * x * r).abs()).sum((0, 1, 2)) + 1e-38)
    a, m = r * w * dy, (w * dy * x).mean(-1, keepdim=True)
    dx = a - x * r ** 3 * m
    m1 = (w * dy * x).abs().mean(-1, keepdim=True)
    em = (w * x).abs().mul(edy).mean(-1, keepdim=True) + (d + 4) * E32 * m1
    e = (r * w).abs() * edy + (x * r ** 3).abs() * em + (3 * er + 8 * E32) * (a.abs() + (x * r ** 3).abs() * m1)
    out["dx"] = (dx, u * (dx.abs() + e) + e + tiny)
    return out


def encode(x):
    """Codes and scales of rows: the quotient as the number it is (a 64-bit
    division of an 18-bit number by an 11-bit one is exact at ties)."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    fine = (top > 0) & torch.isfinite(top)
    code = torch.where(fine, torch.round(127 * x / torch.where(fine, top, 1.0)), 0.0)
    return code.to(torch.int8), (top[..., 0] / 127).float()


def values(code, scale):
    """What codes [slots, 64, hk, d] with scales [slots, hk, 64] stand for, in 64 bits."""
    return code.double() * scale.double().transpose(1, 2)[..., None]


def pool(k, kept):
    """Pooled keys of a block's first `kept` keys k [64, hk, d] in 64 bits."""
    total = k[:kept].sum(0)
    top = total.abs().amax(-1, keepdim=True)
    some = top > 0
    code = torch.where(some, torch.round(total * (127.0 / torch.where(some, top, 1.0))), 0.0).to(torch.int8)
    return code, (top[:, 0] / (127.0 * kept)).float()


def attention(c, q, k, v, w):
    """attn_ref.attention, with what it leaves out of the bound on o: the
    hardware's exp2 gives normal numbers or zero, so a weight, taken relative to
    a score that was the largest (its own weight is 1, and the sum that divides
    at least that), may be off by 2^-126 more."""
    out = A.attention(c, q, k, v, w)
    g = c["hq"] // c["hk"]
    on = (w > 0).double().repeat_interleave(g, 1)
    vt = torch.where((w > 0).any(-2)[..., None], v.permute(0, 2, 1, 3), 0.0).abs().repeat_interleave(g, 1)
    value, bound = out["o"]
    out["o"] = (value, bound + 2.0 ** -126 * (on @ vt).permute(0, 2, 1, 3))
    return out


def attention8(c, q, k, v, w):
    """The same where each weight, times its value's scale, enters as two bf16
    parts: within 2^-16 of itself, and what is below 2^-126 counts as zero (127
    of it at most with the code, against a sum of weights of at least 1).  The
    rest as attn_ref.attention counts it; only the output is rounded to the type."""
    out = A.attention(c, q, k, v, w)
    u, e32 = torch.finfo(c["dtype"]).eps / 2, E32
    g, d, n = c["hq"] // c["hk"], c["d"], c["nk"]
    scale = c.get("scale") or 1.0 / math.sqrt(d)
    on = (w > 0).repeat_interleave(g, 1)
    seen = (w > 0).any(-2)[..., None]
    kt, vt = (torch.where(seen, x.permute(0, 2, 1, 3), 0.0).repeat_interleave(g, 1) for x in (k, v))
    qt = torch.where(on.any(-1)[..., None], q.permute(0, 2, 1, 3), 0.0)
    s = scale * (qt @ kt.transpose(-1, -2)) + torch.log(w.clamp(min=1e-300)).repeat_interleave(g, 1)
    far = torch.where(on, s - torch.where(on.any(-1), out["lse"][0], 0.0)[..., None], -math.inf)
    es = torch.where(on, (d + 2) * e32 * scale * (qt.abs() @ kt.abs().transpose(-1, -2)), 0.0).amax(-1, keepdim=True)
    ew = 2 * es + (24 + n) * e32 + 4 * e32 * torch.where(on, far.abs(), 0.0).amax(-1, keepdim=True)
    value = out["o"][0].permute(0, 2, 1, 3)
    bound = ((u + 4 * e32) * value.abs() + 1.02 * (2.0 ** -16 + ew) * (torch.exp(far) @ vt.abs())
             + 2.0 ** -119 * on.sum(-1, keepdim=True) + 2.0 ** -126 * (on.double() @ vt.abs())
             + torch.finfo(c["dtype"]).smallest_normal * u)
    return {"o": (out["o"][0], bound.permute(0, 2, 1, 3)), "lse": out["lse"]}


def freqs(pairs, base=10000.0):
    return [base ** (-p / max(1, pairs)) for p in range(pairs)]


def rms(x):
    return math.sqrt(x.double().square().mean().item())
