"""Plain attention over listed blocks in 64 bits, with bounds on how far a
kernel may be from it.

The bounds count roundings.  u is half a step of the element type relative to
the value (torch.finfo(t).eps / 2): an output is rounded once, and each weight
p (and its gradient ds) once for the product that takes it.  Scores are sums
of dim products in 32 bits, off by at most (dim + 2) 2^-24 sum |q k| scale; a
score that is off by e moves a weight by e of itself, and the sum it is
divided by as much again.  Sums of n terms in 32 bits add n 2^-24 of the sum
of magnitudes; exp2 and log2 a few steps of 2^-23.

Half a step is relative only down to the type's smallest normal value; below
it a rounding is off by `tiny`, half the spacing of its subnormals (2^-25 for
f16: a correctly rounded gradient of 5.8e-7 is off by 7e-9, more than u of
it), and so is each rounded weight."""
import math

import torch

PAGE = 64


def sees(c, lists, lens, starts, tree, table_ok=None):
    """[b, hk, nq, nk] times each key counts for each query."""
    b, nq, nk, hk = c["b"], c["nq"], c["nk"], c["hk"]
    nkb, nqb = -(-nk // PAGE), -(-nq // c["q_block"])
    out = torch.zeros((b, hk, nq, nk), dtype=torch.float64)
    key = torch.arange(nk)
    for i in range(b):
        n = min(max(int(lens[i]), 0), nk)
        for t in range(nq):
            pos = int(starts[i]) + t
            if pos < 0 or pos >= n:
                continue
            if tree is None:
                m = key <= pos
            else:
                u = key - int(starts[i])
                bits = int(tree[i, t]) & (2 ** 64 - 1)
                m = torch.tensor([int(x) < 0 or (int(x) < 64 and bits >> int(x) & 1) for x in u], dtype=torch.bool)
            m = (m & (key < n)).double()
            for h in range(hk):
                if lists is None:
                    times = torch.ones(nkb)
                else:
                    times = torch.zeros(nkb)
                    for j in lists[i, h, t // c["q_block"]].tolist():
                        if 0 <= j < nkb:
                            times[j] += 1
                if table_ok is not None:
                    times = times * table_ok[i]
                out[i, h, t] = m * times.double()[key // PAGE]
    return out


def attention(c, q, k, v, w, grad=None):
    """o, lse (and dq, dk, dv) with bounds: {name: (value, bound)}.  q [b, nq,
    hq, d], k and v [b, nk, hk, d] in 64 bits; w from sees()."""
    u = torch.finfo(c["dtype"]).eps / 2
    tiny = torch.finfo(c["dtype"]).smallest_normal * u
    g, d = c["hq"] // c["hk"], c["d"]
    scale = c.get("scale") or 1.0 / math.sqrt(d)
    e32 = 2.0 ** -24
    qt = q.permute(0, 2, 1, 3)
    kt = k.permute(0, 2, 1, 3).repeat_interleave(g, 1)
    vt = v.permute(0, 2, 1, 3).repeat_interleave(g, 1)
    w = w.repeat_interleave(g, 1)
    on = w > 0
    clean = on.any(-2)[..., None]  # keys nobody sees may hold anything
    kt, vt = torch.where(clean, kt, 0.0), torch.where(clean, vt, 0.0)
    live = on.any(-1)
    qt = torch.where(live[..., None], qt, 0.0)
    s = scale * (qt @ kt.transpose(-1, -2)) + torch.where(on, torch.log(w.clamp(min=1e-300)), -math.inf)
    lse = torch.logsumexp(s, -1)
    safe = torch.where(live, lse, 0.0)[..., None]
    p = torch.where(on, torch.exp(s - safe), 0.0)
    o = p @ vt
    # scores, weights
    es = (d + 2) * e32 * scale * (qt.abs() @ kt.abs().transpose(-1, -2))
    es = torch.where(on, es, 0.0).amax(-1, keepdim=True)
    n = c["nk"]
    ew = 2 * es + 16 * e32 + (8 + n) * e32 + 4 * e32 * torch.where(on, (s - safe).abs(), 0.0).amax(-1, keepdim=True)
    po = p @ vt.abs()
    bo = (u + 4 * e32) * o.abs() + 1.02 * ((u + ew) * po + tiny * (on.double() @ vt.abs())) + tiny
    out = {"o": (o.permute(0, 2, 1, 3), bo.permute(0, 2, 1, 3)),
           "lse": (lse, (es[..., 0] + (16 + n) * e32 + 8 * e32 * torch.where(live, lse, 0.0).abs()))}
    if grad is None:
        return out
    gt = torch.where(live[..., None], grad.permute(0, 2, 1, 3), 0.0)
    delta = (gt * o).sum(-1, keepdim=True)
    edelta = (gt.abs() * bo).sum(-1, keepdim=True) + (d + 2) * e32 * (gt.abs() * (o.abs() + bo)).sum(-1, keepdim=True)
    dp = gt @ vt.transpose(-1, -2)
    edp = (d + 2) * e32 * (gt.abs() @ vt.abs().transpose(-1, -2))
    ds = p * (dp - delta)
    elp = ew + out["lse"][1][..., None]  # the weights again, from the rounded lse
    eds = tiny * on + 1.02 * ((u + elp) * ds.abs() + p * (1 + elp) * (edp + edelta + 4 * e32 * (dp.abs() + delta.abs())))
    rows = c["nq"] * g

    def per_key(x):
        return x.reshape(x.shape[0], c["hk"], g, *x.shape[2:]).sum(2).permute(0, 2, 1, 3)

    dq, bq = scale * ds @ kt, scale * (eds @ kt.abs() + n * e32 * (ds.abs() @ kt.abs()))
    dk, bk = scale * ds.transpose(-1, -2) @ qt, scale * (eds + rows * e32 * ds.abs()).transpose(-1, -2) @ qt.abs()
    dv, bv = p.transpose(-1, -2) @ gt, 1.02 * ((u + elp + rows * e32) * p + tiny * on).transpose(-1, -2) @ gt.abs()
    dk, bk, dv, bv = per_key(dk), per_key(bk), per_key(dv), per_key(bv)
    dq, bq = dq.permute(0, 2, 1, 3), bq.permute(0, 2, 1, 3)
    for name, x, e in (("dq", dq, bq), ("dk", dk, bk), ("dv", dv, bv)):
        out[name] = (x, (u + 4 * e32) * (x.abs() + e) + e + tiny)
    return out


def check(name, got, value, bound):
    """Every element within its bound; infinities where the value has them."""
    got = got.detach().double().cpu()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    fine = torch.isfinite(value)
    assert torch.equal(torch.isfinite(got), fine), f"{name}: infinities or NaN in other places"
    assert torch.equal(got[~fine], value[~fine]), f"{name}: other infinities"
    off = (got - value).abs()[fine]
    worst = (off / bound[fine]).max().item() if off.numel() else 0.0
    print(f"{name}: worst error {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.3f} times its bound"


def pool(k, lens, nk):
    """Pooled keys of [b, nk, hk, d]: int8 [b, nkb, hk, d], scale [b, nkb, hk]
    (zeros where a block has no key)."""
    b, _, hk, d = k.shape
    nkb = -(-nk // PAGE)
    values = torch.zeros((b, nkb, hk, d), dtype=torch.int8)
    scale = torch.zeros((b, nkb, hk), dtype=torch.float32)
    for i in range(b):
        n = min(max(int(lens[i]), 0), nk)
        for j in range(-(-n // PAGE)):
            x = k[i, j * PAGE:min(n, (j + 1) * PAGE)].double()
            total = x.sum(0)
            top = total.abs().amax(-1, keepdim=True)
            values[i, j] = torch.where(top > 0, torch.round(total * (127.0 / top)), 0.0).to(torch.int8)
            scale[i, j] = (top[:, 0] / (127.0 * x.shape[0])).float()
    return values, scale


def select(c, q, values, scale, lens, starts, sink, local):
    """Lists from pooled keys [b, nkb, hk, d] by the definition."""
    b, nq, hk, g, qb = c["b"], c["nq"], c["hk"], c["hq"] // c["hk"], c["q_block"]
    nqb, keep = -(-nq // qb), c["blocks"]
    lists = torch.full((b, hk, nqb, keep), -1, dtype=torch.int32)
    for i in range(b):
        n = min(max(int(lens[i]), 0), c["nk"])
        for y in range(nqb):
            ts = [t for t in range(y * qb, min(nq, (y + 1) * qb)) if 0 <= int(starts[i]) + t < n]
            if not ts:
                continue
            count = (int(starts[i]) + ts[-1]) // PAGE + 1
            for h in range(hk):
                total = q[i, ts, h * g:(h + 1) * g].double().sum((0, 1))
                top = total.abs().max()
                q8 = torch.round(total * (127.0 / top)) if top > 0 else torch.zeros_like(total)
                score = (values[i, :count, h].double() @ q8).float() * scale[i, :count, h] + 0.0
                order = sorted(range(count), key=lambda j: (not (j < sink or j >= count - local), -float(score[j]), j))
                best = sorted(order[:keep])
                lists[i, h, y, :len(best)] = torch.tensor(best, dtype=torch.int32)
    return lists
