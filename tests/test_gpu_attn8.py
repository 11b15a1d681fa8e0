"""What stands around attention over a cache, on the GPU against plain forms in
64 bits (attn8_ref.py, attn_ref.py), whose bounds count roundings."""
import math

import numpy as np
import pytest
import torch

import attn8_ref as R
import attn_ref as A
from test_gpu_attn import case, plan, poison, random_lists

pytestmark = pytest.mark.gpu
PAGE = 64
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def S():
    import sparse_dense_matrix_amd as S
    assert torch.cuda.is_available()
    return S


def kind(S, dtype):
    return S.BF16 if dtype == BF else S.F16


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- norm and rotation -----------------------------------------------------

def rope_case(b=1, n=1, hq=2, hk=1, d=64, dtype=BF, pairs=None, axes=1, interleaved=False, norm=True, eps=1e-6,
              lens=None, starts=None):
    return dict(b=b, n=n, hq=hq, hk=hk, d=d, dtype=dtype, pairs=d // 2 if pairs is None else pairs, axes=axes,
                interleaved=interleaved, norm=norm, eps=eps, lens=lens, starts=starts)


ROPE = [
    rope_case(), rope_case(b=3, n=5, hq=5, hk=5, d=128, interleaved=True),
    rope_case(b=2, n=33, hq=12, hk=4, d=128, dtype=HF, pairs=16), rope_case(n=129, hq=6, hk=2, pairs=24, axes=3, interleaved=True),
    rope_case(n=70, hq=16, hk=1, d=128, pairs=0), rope_case(b=2, n=7, hq=3, hk=3, norm=False, dtype=HF),
    rope_case(b=4, n=9, hq=32, hk=8, d=128, lens=[9, 0, 4, 100], starts=[0, 0, -2, 95]),
    rope_case(b=32, n=1, hq=32, hk=8, d=128, starts=[1000 * i for i in range(32)]),
    rope_case(b=3, n=2, starts=[2 ** 31 - 2, -2 ** 31, 1048576], d=128, eps=0.0),
    rope_case(n=5000, hq=1, hk=1, pairs=8), rope_case(b=2, n=40, axes=2, pairs=32, d=128, dtype=HF),
]


def rope_plan(S, c, **kw):
    return S.spmm_plan_attn_rope(c["b"], c["n"], c["hq"], c["hk"], c["d"], R.freqs(c["pairs"]), axis=axis_of(c),
                                 axes=c["axes"], dtype=kind(S, c["dtype"]), interleaved=c["interleaved"], eps=c["eps"], **kw)


def axis_of(c):
    return [p * c["axes"] // c["pairs"] for p in range(c["pairs"])]


def rope_inputs(c, seed):
    g = torch.Generator().manual_seed(seed)

    def make(h):
        scale = torch.exp(torch.randn((c["b"], c["n"], h, 1), generator=g))
        return (torch.randn((c["b"], c["n"], h, c["d"]), generator=g) * scale).to(c["dtype"])

    q, k, gq, gk = make(c["hq"]), make(c["hk"]), make(c["hq"]), make(c["hk"])
    w = 1 + 0.3 * torch.randn((2, c["d"]), generator=g) if c["norm"] else (None, None)
    place = torch.randint(-100, 100000, (c["axes"], c["b"], c["n"]), generator=g).int() if c["axes"] > 1 else None
    pos, alive = R.live(c["b"], c["n"], c["lens"], c["starts"] or [0] * c["b"])
    at = pos[None] if place is None else place.long()
    return q, k, gq, gk, w[0], w[1], place, alive, *R.angles(R.freqs(c["pairs"]), axis_of(c), at)


def cuda(x):
    return None if x is None else x.cuda()


@pytest.mark.parametrize("n", range(len(ROPE)))
def test_rope(S, n):
    c = ROPE[n]
    q, k, gq, gk, qw, kw, place, alive, angle, off = rope_inputs(c, 300 + n)
    dead = ~alive[..., None, None]
    for x in (q, k, gq, gk):  # what no live token uses may hold anything
        x.masked_fill_(dead, float("nan"))
    P = rope_plan(S, c, backward=True)
    at = dict(q_weight=cuda(qw), k_weight=cuda(kw), positions=cuda(place), lens=ints(c["lens"]), starts=ints(c["starts"]))
    qo, ko = torch.full_like(q, 7.0).cuda(), torch.full_like(k, 7.0).cuda()
    S.spmm_execute_attn_rope(P, q.cuda(), k.cuda(), qo, ko, **at)
    dq, dk = poison(q).cuda(), poison(k).cuda()
    dqw, dkw = torch.full((2, c["d"]), float("nan"), device="cuda") if c["norm"] else (None, None)
    S.spmm_execute_attn_rope_backward(P, gq.cuda(), gk.cuda(), cuda(q if c["norm"] else None), cuda(k if c["norm"] else None),
                                      dq, dk, dq_weight=dqw, dk_weight=dkw, **at)
    for name, x, w, grad, o, dx, dw in (("q", q, qw, gq, qo, dq, dqw), ("k", k, kw, gk, ko, dk, dkw)):
        want = R.rope(torch.where(dead, 0.0, x.double()), None if w is None else w.double(), angle, off, c["interleaved"],
                      c["eps"], c["dtype"], torch.where(dead, 0.0, grad.double()), alive)
        value, bound = want["o"]
        A.check(name, o, torch.where(dead, 7.0, value), bound)  # the others stay as they were
        A.check("d" + name, dx, *want["dx"])
        if w is not None:
            A.check(f"d{name}_weight", dw, *want["dw"])


# rows enough for the kernels of many: tokens in groups of 16 (up to 16 heads) and of 4
MANY = [rope_case(b=2, n=2500, hq=12, hk=4, pairs=24, interleaved=True, lens=[2500, 1777], starts=[0, -3]),
        rope_case(n=5003, hq=9, hk=5, d=128, dtype=HF, axes=2), rope_case(b=3, n=701, hq=32, hk=8, d=128, pairs=40),
        rope_case(b=2, n=1399, hq=20, hk=20, dtype=HF, lens=[0, 1399], starts=[5, 40], interleaved=True),
        rope_case(b=67, n=29, hq=33, hk=2, norm=False, starts=[100 * i for i in range(67)])]


@pytest.mark.parametrize("n", range(len(MANY)))
def test_rope_of_many_rows(S, n):
    """Against the plain form, as above, and token by token: a short call on the
    same tokens (another kernel) gives the same bits."""
    c = MANY[n]
    q, k, _, _, qw, kw, place, alive, angle, off = rope_inputs(c, 600 + n)
    w = {} if qw is None else dict(q_weight=qw.cuda(), k_weight=kw.cuda())
    positions = place.to(torch.int32).cuda() if c["axes"] > 1 else None
    qo, ko = torch.full_like(q, 7.0).cuda(), torch.full_like(k, 7.0).cuda()
    S.spmm_execute_attn_rope(rope_plan(S, c), q.cuda(), k.cuda(), qo, ko, positions=positions, lens=ints(c["lens"]),
                             starts=ints(c["starts"]), **w)
    dead = ~alive[:, :, None, None]
    for name, x, o, wt in (("q", q, qo, qw), ("k", k, ko, kw)):
        value, bound = R.rope(torch.where(dead, 0.0, x.double()), None if wt is None else wt.double(), angle, off,
                              c["interleaved"], c["eps"], c["dtype"])["o"]
        A.check(name, o, torch.where(dead, 7.0, value), bound)
    short = dict(c, n=5)
    first = c["n"] - 5
    few = rope_plan(S, short)
    x, y = (t[:, first:].contiguous().cuda() for t in (q, k))
    qs, ks = torch.full_like(x, 7.0), torch.full_like(y, 7.0)
    S.spmm_execute_attn_rope(few, x, y, qs, ks, positions=None if positions is None else positions[:, :, first:].contiguous(),
                             lens=ints(c["lens"]), starts=ints([s + first for s in c["starts"] or [0] * c["b"]]), **w)
    assert torch.equal(qs, qo[:, first:]) and torch.equal(ks, ko[:, first:])


def test_rope_in_place_and_packed(S):
    """q, k of one packed buffer, turned in place, and gradients over their own inputs."""
    c = rope_case(b=2, n=37, hq=6, hk=2, d=128)
    q, k, gq, gk, qw, kw, *_ = rope_inputs(c, 1)
    P = rope_plan(S, c, backward=True)
    w = dict(q_weight=qw.cuda(), k_weight=kw.cuda())
    qo, ko = torch.empty_like(q).cuda(), torch.empty_like(k).cuda()
    S.spmm_execute_attn_rope(P, q.cuda(), k.cuda(), qo, ko, **w)
    packed = torch.cat((q, k, k), 2).cuda()
    a, b, v = packed.split((6, 2, 2), 2)
    S.spmm_execute_attn_rope(P, a, b, a, b, **w)
    assert torch.equal(a, qo) and torch.equal(b, ko) and torch.equal(v, k.cuda())
    outs = []
    for own in (False, True):
        grads = torch.cat((gq, gk), 2).cuda()
        g1, g2 = grads.split((6, 2), 2)
        dq, dk = (g1, g2) if own else (torch.empty_like(q).cuda(), torch.empty_like(k).cuda())
        dw = torch.empty((2, 128), device="cuda")
        S.spmm_execute_attn_rope_backward(P, g1, g2, q.cuda(), k.cuda(), dq, dk, dq_weight=dw[0], dk_weight=dw[1], **w)
        outs.append((dq.clone(), dk.clone(), dw))
    assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_rope_one_weight_and_broadcast_gradient(S):
    """A norm for the queries alone; one gradient for all heads."""
    c = rope_case(b=2, n=19, hq=4, hk=2)
    q, k, gq, gk, qw, _, _, alive, angle, off = rope_inputs(c, 2)
    P = rope_plan(S, c, backward=True)
    dq, dk, dw = poison(q).cuda(), poison(k).cuda(), torch.empty(64, device="cuda")
    g1 = gq[:, :, :1].cuda().expand(-1, -1, 4, -1)
    S.spmm_execute_attn_rope_backward(P, g1, gk.cuda(), q.cuda(), None, dq, dk, q_weight=qw.cuda(), dq_weight=dw)
    want = R.rope(q.double(), qw.double(), angle, off, False, 1e-6, BF, g1.cpu().double(), alive)
    A.check("dq", dq, *want["dx"])
    A.check("dw", dw, *want["dw"])
    A.check("dk", dk, *R.rope(k.double(), None, angle, off, False, 1e-6, BF, gk.double(), alive)["dx"])


def test_rope_spreads_nothing_between_rows(S):
    c = rope_case(n=9, hq=3, hk=1, d=128, dtype=HF)
    q, k, *_, qw, kw, _, _, _, _ = rope_inputs(c, 3)
    P = rope_plan(S, c)
    outs = []
    for bad in (False, True):
        if bad:
            q[0, 4, 1, 5], k[0, 2, 0, 100] = float("inf"), float("nan")
        qo, ko = torch.zeros_like(q).cuda(), torch.zeros_like(k).cuda()
        S.spmm_execute_attn_rope(P, q.cuda(), k.cuda(), qo, ko, q_weight=qw.cuda(), k_weight=kw.cuda())
        outs.append((qo, ko))
    same = outs[0][0] == outs[1][0]
    same[0, 4, 1] = True
    assert same.all() and torch.equal(torch.isnan(outs[1][1]).any(-1)[0, :, 0].cpu(), torch.arange(9) == 2)


def test_rope_without_tokens(S):
    P = rope_plan(S, rope_case(b=0, n=4), backward=True)
    q, k, w = torch.empty((0, 4, 2, 64), dtype=BF, device="cuda"), torch.empty((0, 4, 1, 64), dtype=BF, device="cuda"), \
        torch.ones(64, device="cuda")
    S.spmm_execute_attn_rope(P, q, k, q, k, q_weight=w, k_weight=w)
    dw = torch.full((2, 64), float("nan"), device="cuda")
    S.spmm_execute_attn_rope_backward(P, q, k, q, k, q, k, q_weight=w, k_weight=w, dq_weight=dw[0], dk_weight=dw[1])
    assert (dw == 0).all()


# ---- the cache -------------------------------------------------------------

def empty_cache(pages, hk, d, fill=99):
    k8, v8 = torch.full((2, pages, PAGE, hk, d), fill, dtype=torch.int8, device="cuda")
    ks, vs = torch.full((2, pages, hk, PAGE), float("nan"), device="cuda")
    return k8, v8, ks, vs


def rows(shape, dtype, g):
    """Rows of uneven size, some zero, some with ties, some near the type's ends."""
    x = torch.randn(shape, generator=g) * torch.exp(2 * torch.randn((*shape[:-1], 1), generator=g))
    kind_of = torch.randint(0, 12, (*shape[:-1], 1), generator=g)
    ties = torch.randint(-127, 128, shape, generator=g) / 2
    ties[..., 3] = 127.0
    x = torch.where(kind_of == 0, 0.0, torch.where(kind_of == 1, ties, x))
    x = torch.where(kind_of == 2, x * torch.finfo(dtype).smallest_normal / 8, x).clamp(-6e4, 6e4)
    return x.to(dtype)


WRITE = [dict(b=1, n=1, nk=64), dict(b=3, n=5, nk=200, hk=3, d=128), dict(b=2, n=130, nk=130, dtype=HF),
         dict(b=40, n=1, nk=1000, hk=8, d=128), dict(b=1, n=1000, nk=1000, hk=1, dtype=HF, d=128),
         dict(b=3, n=1500, nk=1601, hk=8, dtype=HF, d=128), dict(b=2, n=2100, nk=2100, hk=8)]  # enough to go by blocks


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("n", range(len(WRITE)))
def test_write_and_read(S, n, paged):
    c = {"hk": 2, "d": 64, "dtype": BF, **WRITE[n]}
    b, nq, nk, hk, d = c["b"], c["n"], c["nk"], c["hk"], c["d"]
    nkb = -(-nk // PAGE)
    g = torch.Generator().manual_seed(400 + n)
    k, v = rows((b, nq, hk, d), c["dtype"], g), rows((b, nq, hk, d), c["dtype"], g)
    k[0, 0, 0, 1], v[-1, -1, -1, 0] = float("nan"), float("-inf")
    lens = [max(0, nk + 3 - 7 * i) if i != 1 else nk // 2 for i in range(b)]
    starts = [min(max(0, n_i - nq), nk - nq) + (-1 if i == 2 else i % 2) for i, n_i in enumerate(lens)]
    table = None
    if paged:
        table = torch.randperm(b * nkb + 2, generator=g)[:b * nkb].reshape(b, nkb).int()
        if b > 1:
            table[1, 0], table[-1, -1] = -5, b * nkb + 2  # no pages
    pages = b * nkb + 2
    P = S.spmm_plan_attn(b, nq, nk, hk, hk, d, dtype=kind(S, c["dtype"]))
    k8, v8, ks, vs = empty_cache(pages if paged else b * nkb, hk, d)
    if not paged:
        k8, v8 = (x.reshape(b, -1, hk, d)[:, :nk] for x in (k8, v8))  # rows of whole blocks, the last cut off
    want = [x.clone().cpu() for x in (k8, v8, ks, vs)]
    S.spmm_execute_attn_write(P, k.cuda(), v.cuda(), k8, v8, ks, vs, table=cuda(table), lens=ints(lens), starts=ints(starts))
    there = torch.zeros((b, nk), dtype=torch.bool)
    for i in range(b):
        for t in range(nq):
            pos = starts[i] + t
            if not 0 <= pos < min(lens[i], nk):
                continue
            slot = int(table[i, pos // PAGE]) if paged else i * nkb + pos // PAGE
            if not 0 <= slot < pages:
                continue
            there[i, pos] = True
            for x, code, scale in ((k, 0, 2), (v, 1, 3)):
                where = (slot, pos % PAGE) if paged else (i, pos)
                want[code][where], want[scale][slot, :, pos % PAGE] = R.encode(x[i, t])
    for got, w in zip((k8, v8, ks, vs), want):
        assert torch.equal(torch.nan_to_num(got.cpu().float(), 1e30, 2e30), torch.nan_to_num(w.float(), 1e30, 2e30))
    # read back: positions below the length, zeros where there is no page
    kr, vr = torch.full((2, b, nk, hk, d), 3.0, dtype=c["dtype"], device="cuda")
    S.spmm_execute_attn_read(P, k8, v8, ks, vs, kr, vr, table=cuda(table), lens=ints(lens))
    u = torch.finfo(c["dtype"]).eps / 2
    for got, code, scale in ((kr, 0, 2), (vr, 1, 3)):
        got = got.cpu().double()
        value = got.clone()  # places nothing was written to may hold anything
        for i in range(b):
            n_i = min(lens[i], nk)
            value[i, n_i:] = 3.0
            for pos in range(n_i):
                slot = int(table[i, pos // PAGE]) if paged else i * nkb + pos // PAGE
                if not 0 <= slot < pages:
                    value[i, pos] = 0.0
                elif there[i, pos]:
                    value[i, pos] = want[code][(slot, pos % PAGE) if paged else (i, pos)].double() * \
                        want[scale][slot, :, pos % PAGE].double()[:, None]
        assert torch.equal(got.isnan(), value.isnan())
        got, value = torch.nan_to_num(got), torch.nan_to_num(value)
        # the product is rounded to 32 bits, then to the type
        A.check("read", got, value, (u + 2 * R.E32) * value.abs() + torch.finfo(c["dtype"]).smallest_normal * u)


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("n", [66, 1500])
def test_write_of_sequences_far_from_their_keys(S, n, paged):
    """Positions at the ends of 32 bits, as idle sequences may have: nothing of
    theirs is read or written, in the kernel that goes by blocks and the other."""
    starts = [-2 ** 31, -2 ** 31 + 61, 2 ** 31 - 1, 100, 2 ** 31 - 65, -n + 30, 2 ** 31 - 129]
    b, nk, hk, d = len(starts), 4096, 8 if n == 1500 else 72, 64
    nkb = nk // PAGE
    g = torch.Generator().manual_seed(450)
    k, v = rows((b, n, hk, d), BF, g), rows((b, n, hk, d), BF, g)
    for i in (0, 1, 2, 4, 6):
        k[i], v[i] = float("nan"), float("nan")
    lens = [nk, nk, nk, nk, 10, nk, 0]
    table = torch.randperm(b * nkb, generator=g).reshape(b, nkb).int() if paged else None
    cache = empty_cache(b * nkb, hk, d)
    want = [x.clone() for x in cache]
    k8, v8, ks, vs = cache
    if not paged:
        k8, v8 = (x.view(b, nk, hk, d) for x in (k8, v8))
    P = S.spmm_plan_attn(b, n, nk, hk, hk, d)
    S.spmm_execute_attn_write(P, k.cuda(), v.cuda(), k8, v8, ks, vs, table=cuda(table), lens=ints(lens), starts=ints(starts))
    for i, first, t in ((3, 100, 0), (5, 0, n - 30)):  # positions from `first` on, of tokens from t on
        pos = torch.arange(first, first + n - t)
        slot = table[i, pos // PAGE].long() if paged else i * nkb + pos // PAGE
        for x, code, scale in ((k, 0, 2), (v, 1, 3)):
            c, f = R.encode(x[i, t:])
            want[code][slot.cuda(), (pos % PAGE).cuda()] = c.cuda()
            want[scale][slot.cuda(), :, (pos % PAGE).cuda()] = f.cuda()
    for got, w in zip(cache, want):
        assert torch.equal(torch.nan_to_num(got.float(), 1e30), torch.nan_to_num(w.float(), 1e30))


def test_codes_of_every_value(S):
    """Each finite bf16 number next to each of a few tops: the code is the rounded quotient's."""
    bits = torch.arange(-2 ** 15, 2 ** 15).short()
    x = bits.view(BF)
    x = x[torch.isfinite(x)]
    for top in (1.0, 127.0, 2.0 ** -126, 3.3e38, 0.7578125, 1.984375, 2.0 ** -121, 2.0 ** -133, 2.0 ** 120, 2.0 ** 127):
        keep = x[x.abs() <= torch.tensor(top).to(BF)]
        keep = keep[:keep.numel() // 63 * 63].reshape(-1, 63)
        r = torch.cat((keep, torch.full((keep.shape[0], 1), top).to(BF)), 1)
        n = r.shape[0]
        r = r.reshape(1, n, 1, 64)
        P = S.spmm_plan_attn(1, n, n, 1, 1, 64)
        k8, v8, ks, vs = empty_cache(-(-n // PAGE), 1, 64)
        k8, v8 = k8.reshape(1, -1, 1, 64)[:, :n], v8.reshape(1, -1, 1, 64)[:, :n]
        S.spmm_execute_attn_write(P, r.cuda(), r.cuda(), k8, v8, ks, vs)
        code, scale = R.encode(r)
        assert torch.equal(k8.cpu(), code) and torch.equal(v8.cpu(), code)
        assert torch.equal(ks.reshape(-1)[:n].cpu(), scale.reshape(-1))


def test_codes_of_ties(S):
    """fp16 rows whose quotients are half a whole number: the even code."""
    for e in range(-24, 9):
        top = 254.0 * 2.0 ** e
        x = torch.arange(-254, 255, 2)[:252].float() * 0.5 * 2.0 ** (e + 1)
        x = torch.stack((x + 2.0 ** e, x)).reshape(-1, 63)
        r = torch.cat((x, torch.full((x.shape[0], 1), top)), 1).to(HF)
        n = r.shape[0]
        r = r.reshape(1, n, 1, 64)
        P = S.spmm_plan_attn(1, n, n, 1, 1, 64, dtype=S.F16)
        k8, v8, ks, vs = empty_cache(1, 1, 64)
        k8, v8 = k8.reshape(1, -1, 1, 64)[:, :n], v8.reshape(1, -1, 1, 64)[:, :n]
        S.spmm_execute_attn_write(P, r.cuda(), r.cuda(), k8, v8, ks, vs)
        code, scale = R.encode(r)
        assert torch.equal(k8.cpu(), code) and torch.equal(v8.cpu(), code)
        assert torch.equal(ks.reshape(-1)[:n].cpu(), scale.reshape(-1))


def filled(S, c, g, pages=None, far=0):
    """A cache of random rows through a random table, what its codes stand for
    as [b, nk, hk, d] in 64 bits, and the table."""
    b, nk, hk, d = c["b"], c["nk"], c["hk"], c["d"]
    nkb = -(-nk // PAGE)
    pages = pages or b * nkb + 1
    table = torch.randperm(pages, generator=g)[:b * nkb].reshape(b, nkb).int()
    out = []
    for _ in range(2):
        x = torch.randn((pages, PAGE, hk, d), generator=g) * torch.exp(torch.randn((pages, PAGE, hk, 1), generator=g))
        code, scale = R.encode(x.to(c["dtype"]))
        out.append((code, scale.transpose(1, 2).contiguous()))
    at = table.long()
    k, v = (R.values(code, scale)[at].flatten(1, 2)[:, :nk] for code, scale in out)
    return [x.cuda() for x in (out[0][0], out[1][0], out[0][1], out[1][1])], k, v, table


POOL = [dict(b=1, nk=64), dict(b=3, nk=200, hk=3, d=128), dict(b=2, nk=1000, hk=8, d=128, nq=70), dict(b=5, nk=130, hk=1),
        dict(b=3, nk=6500, nq=6500, hk=7), dict(b=2, nk=8190, nq=8190, hk=9, d=128)]  # blocks enough for a wave each


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("n", range(len(POOL)))
def test_pool8(S, n, paged):
    c = {"hk": 2, "d": 64, "dtype": BF, "nq": 1, **POOL[n]}
    g = torch.Generator().manual_seed(500 + n)
    (k8, _, ks, _), k, _, table = filled(S, c, g)
    b, nk, hk, d = c["b"], c["nk"], c["hk"], c["d"]
    nkb = -(-nk // PAGE)
    lens = [nk, nk // 2, 0, nk + 9, 1][:b]
    first = [max(0, n_i - c["nq"]) for n_i in lens]
    P = S.spmm_plan_attn(b, c["nq"], nk, hk, hk, d)
    pages = k8.shape[0]
    if not paged:  # sequences side by side
        k8 = k8[table.long().cuda()].flatten(1, 2)[:, :nk].contiguous()
        ks = ks[table.long().cuda()].flatten(0, 1).contiguous()
        pages = b * nkb
    else:
        table[0, -1] = -1
    pooled, scale = torch.full((pages, hk, d), 7, dtype=torch.int8, device="cuda"), torch.full((pages, hk), 7.0, device="cuda")
    S.spmm_execute_attn_pool8(P, k8, ks, pooled, scale, table=cuda(table) if paged else None, lens=ints(lens), first=ints(first))
    want, want_scale = torch.full((pages, hk, d), 7, dtype=torch.int8), torch.full((pages, hk), 7.0)
    for i in range(b):
        n_i = min(lens[i], nk)
        for j in range(first[i] // PAGE, -(-n_i // PAGE)):
            slot = int(table[i, j]) if paged else i * nkb + j
            if 0 <= slot:
                want[slot], want_scale[slot] = R.pool(k[i, j * PAGE:(j + 1) * PAGE], min(PAGE, n_i - j * PAGE))
    assert torch.equal(pooled.cpu(), want) and torch.equal(scale.cpu(), want_scale)


# ---- attention over it -----------------------------------------------------

CACHE = [
    case(nq=1, nk=1, blocks=1), case(nq=1, nk=65, hq=8, hk=1, d=128), case(b=3, nq=1, nk=4097, hq=8, hk=2, d=128),
    case(b=2, nq=3, nk=200, hq=15, hk=3, dtype=HF), case(nq=1, nk=1000, hq=32, hk=2, d=128, dtype=HF),
    case(b=2, nq=7, nk=333, hq=8, hk=2, d=128), case(nq=5, nk=640, hq=6, hk=1), case(nq=24, nk=777, hq=8, hk=4, d=128),
    case(b=2, nq=40, nk=500, hq=4, hk=2, dtype=HF, d=128), case(nq=64, nk=1500, hq=4, hk=1, d=64),
    case(nq=150, nk=300, hq=4, hk=2, d=128), case(nq=64, nk=3000, hq=16, hk=2, d=128, scale=0.2), case(b=2, nq=33, nk=900, hq=12, hk=1),
    case(nq=2, nk=20000, hq=4, hk=1, d=64), case(nq=9, nk=129, hq=7, hk=7, d=128, dtype=HF),
]


def outputs(c):
    return (torch.full((c["b"], c["nq"], c["hq"], c["d"]), float("nan"), dtype=c["dtype"], device="cuda"),
            torch.full((c["b"], c["hq"], c["nq"]), float("nan"), device="cuda"))


def new_tokens(c, how):
    b, nq, nk = c["b"], c["nq"], c["nk"]
    if how == "full":
        return [nk] * b, [nk - nq] * b
    lens = [max(0, nk - 37 * (i + 1) * nk // 100) for i in range(b)]
    return lens, [n - nq if i % 2 == 0 else n - nq // 2 for i, n in enumerate(lens)]  # some before, some past the keys


@pytest.mark.parametrize("how", ["full", "ragged"])
@pytest.mark.parametrize("n", range(len(CACHE)))
def test_cache8(S, n, how):
    c = CACHE[n]
    g = torch.Generator().manual_seed(600 + n)
    cache, k, v, table = filled(S, c, g)
    q = torch.randn((c["b"], c["nq"], c["hq"], c["d"]), generator=g).to(c["dtype"])
    lens, starts = new_tokens(c, how)
    o, lse = outputs(c)
    S.spmm_execute_attn_cache8(plan(S, c), q.cuda(), *cache, o, lse, table=table.cuda(), lens=ints(lens), starts=ints(starts))
    want = R.attention(c, q.double(), k, v, A.sees(c, None, lens, starts, None))
    A.check("o", o, *want["o"])
    A.check("lse", lse, *want["lse"])


@pytest.mark.parametrize("n", [3, 7, 8, 9])
def test_cache8_tree(S, n):
    c = CACHE[n]
    g = torch.Generator().manual_seed(700 + n)
    cache, k, v, table = filled(S, c, g)
    q = torch.randn((c["b"], c["nq"], c["hq"], c["d"]), generator=g).to(c["dtype"])
    tree = torch.randint(-2 ** 63, 2 ** 63 - 1, (c["b"], c["nq"]), generator=g)
    lens = [c["nk"] - 20 * i for i in range(c["b"])]
    starts = [n_i - c["nq"] for n_i in lens]
    o, lse = outputs(c)
    S.spmm_execute_attn_cache8(plan(S, c), q.cuda(), *cache, o, lse, table=table.cuda(), tree=tree.cuda(), lens=ints(lens),
                               starts=ints(starts))
    want = R.attention(c, q.double(), k, v, A.sees(c, None, lens, starts, tree))
    A.check("o", o, *want["o"])
    A.check("lse", lse, *want["lse"])


@pytest.mark.parametrize("n", [1, 3, 6, 9, 10])
def test_cache8_lists(S, n):
    """Listed blocks, empty lists, blocks without a page, with and without a table."""
    c = dict(CACHE[n], blocks=3, q_block=[64, 16, 4, 1][n % 4])
    g = torch.Generator().manual_seed(800 + n)
    cache, k, v, table = filled(S, c, g)
    q = torch.randn((c["b"], c["nq"], c["hq"], c["d"]), generator=g).to(c["dtype"])
    lists = random_lists(c, g, empty=0.2)
    lens, starts = new_tokens(c, "full")
    outs = []
    for paged in (True, False):
        o, lse = outputs(c)
        k8, v8, ks, vs = cache
        if not paged:
            at = table.long().cuda()
            k8, v8 = (x[at].flatten(1, 2)[:, :c["nk"]].contiguous() for x in (k8, v8))
            ks, vs = (x[at].flatten(0, 1).contiguous() for x in (ks, vs))
        S.spmm_execute_attn_cache8(plan(S, c), q.cuda(), k8, v8, ks, vs, o, lse, table=table.cuda() if paged else None,
                                   lists=lists.cuda(), lens=ints(lens), starts=ints(starts))
        outs.append((o, lse))
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    want = R.attention(c, q.double(), k, v, A.sees(c, lists, lens, starts, None))
    A.check("o", o, *want["o"])
    A.check("lse", lse, *want["lse"])
    bad = table.clone()
    bad[:, 0] = -1
    ok = torch.ones(table.shape)
    ok[:, 0] = 0
    S.spmm_execute_attn_cache8(plan(S, c), q.cuda(), *cache, o, lse, table=bad.cuda(), lists=lists.cuda(), lens=ints(lens),
                               starts=ints(starts))
    want = R.attention(c, q.double(), k, v, A.sees(c, lists, lens, starts, None, ok))
    A.check("o", o, *want["o"])
    A.check("lse", lse, *want["lse"])


@pytest.mark.parametrize("hq,dtype,d", [(8, BF, 64), (40, BF, 128), (40, HF, 64), (16, HF, 128)])
def test_cache8_many_lists(S, hq, dtype, d):
    """Lists enough for a wave each: those of every query of a prompt over a cache."""
    c = case(b=2, nq=1100, nk=1200, hq=hq, hk=2, d=d, dtype=dtype, q_block=1, blocks=2)
    g = torch.Generator().manual_seed(850 + hq + d)
    cache, k, v, table = filled(S, c, g)
    q = torch.randn((2, 1100, hq, d), generator=g).to(dtype)
    lists = random_lists(c, g, empty=0.1)
    lens, starts = [1200, 900], [100, -20]
    o, lse = outputs(c)
    S.spmm_execute_attn_cache8(plan(S, c), q.cuda(), *cache, o, lse, table=table.cuda(), lists=lists.cuda(), lens=ints(lens),
                               starts=ints(starts))
    # the same lists' queries one by one, in 64 bits: 300 of them
    pick = torch.randint(0, 1100, (300,), generator=g).sort().values
    for i in range(2):
        for t in pick.tolist():
            pos = starts[i] + t
            for h in range(2):
                ids = [j for j in lists[i, h, t].tolist() if j >= 0]
                key = torch.cat([torch.arange(j * PAGE, min((j + 1) * PAGE, 1200)) for j in ids] or [torch.zeros(0).long()])
                key = key[(key <= pos) & (key < lens[i])] if 0 <= pos < lens[i] else key[:0]
                heads = slice(h * hq // 2, (h + 1) * hq // 2)
                if not len(key):
                    assert (o[i, t, heads] == 0).all() and (lse[i, heads, t] == -math.inf).all()
                    continue
                sub = dict(b=1, nq=1, nk=len(key), hq=hq // 2, hk=1, d=d, dtype=dtype, q_block=1)
                w = torch.ones((1, 1, 1, len(key)), dtype=torch.float64)
                want = R.attention(sub, q[i:i + 1, t:t + 1, heads].double(), k[i:i + 1, key, h:h + 1], v[i:i + 1, key, h:h + 1], w)
                for got, (value, bound) in ((o[i:i + 1, t:t + 1, heads], want["o"]), (lse[i:i + 1, heads, t:t + 1], want["lse"])):
                    worst = ((got.cpu().double() - value).abs() / bound).max().item()
                    assert worst <= 1, (i, t, h, worst)


@pytest.mark.parametrize("n", [2, 4, 7, 9])
def test_cache8_ignores_what_stands_past_the_length(S, n):
    """Codes past the length are any, scales NaN and infinite: in every kernel."""
    c = CACHE[n]
    g = torch.Generator().manual_seed(900 + n)
    cache, k, v, table = filled(S, c, g)
    q = torch.randn((c["b"], c["nq"], c["hq"], c["d"]), generator=g).to(c["dtype"])
    lens, starts = new_tokens(c, "ragged")
    starts = [n_i - c["nq"] for n_i in lens]
    outs = []
    for spoil in (False, True):
        if spoil:
            for i, n_i in enumerate(lens):
                for pos in range(max(0, n_i), -(-c["nk"] // PAGE) * PAGE):
                    page = int(table[i, pos // PAGE])
                    cache[2][page, :, pos % PAGE], cache[3][page, :, pos % PAGE] = float("nan"), float("inf")
                    cache[0][page, pos % PAGE] = -128
        o, lse = outputs(c)
        S.spmm_execute_attn_cache8(plan(S, c), q.cuda(), *cache, o, lse, table=table.cuda(), lens=ints(lens), starts=ints(starts))
        outs.append((o, lse))
    assert all(torch.equal(x, y) for x, y in zip(*outs)) and not outs[1][0].isnan().any()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq,nq", [(4, 1), (32, 1), (8, 24)])
def test_cache8_values_of_any_size(S, dtype, hq, nq):
    """Values from the type's smallest to its largest, keys that set scores far apart."""
    c = case(nq=nq, nk=512, hq=hq, hk=1, d=128, dtype=dtype)
    g = torch.Generator().manual_seed(31)
    cache, k, v, table = filled(S, c, g)
    big = 6e4 if dtype == HF else 1e30
    size = torch.exp2(torch.linspace(-20, 0, 512)) * big / 127
    size = size[torch.randperm(512, generator=g)]
    at = table.long()[0]
    cache[3][at.cuda()] = size.reshape(8, 1, PAGE).cuda()
    v = cache[1].cpu()[at].reshape(1, 512, 1, 128).double() * size.double()[None, :, None, None]
    grow = torch.linspace(0.01, 0.5, 512)[torch.randperm(512, generator=g)]
    cache[2][at.cuda()] = grow.reshape(8, 1, PAGE).cuda()
    k = cache[0].cpu()[at].reshape(1, 512, 1, 128).double() * grow.double()[None, :, None, None]
    q = torch.randn((1, nq, hq, 128), generator=g).to(dtype)
    o, lse = outputs(c)
    S.spmm_execute_attn_cache8(plan(S, c), q.cuda(), *cache, o, lse, table=table.cuda(), starts=ints([512 - nq]))
    want = R.attention(c, q.double(), k, v, A.sees(c, None, [512], [512 - nq], None))
    A.check("o", o, *want["o"])
    A.check("lse", lse, *want["lse"])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq", [1, 12])
def test_cache8_large_values_that_few_rows_see(S, dtype, hq):
    """Values near the type's end: at a drafted token that only the last row sees,
    and at a key whose weight is about 2^-60, read before the others.  The other
    rows' values are 2^-28 of it, and come out as if it were not there."""
    c = case(nq=24, nk=700, hq=hq, hk=1, d=128, dtype=dtype)
    g = torch.Generator().manual_seed(33)
    cache, _, _, table = filled(S, c, g)
    at = table.long()[0]
    slots = at.repeat_interleave(PAGE)[:700], torch.arange(700) % PAGE
    ks, vs = torch.full((700,), 1 / 700.0), torch.full((700,), 500.0 * 2.0 ** -28)
    vs[[3, 699]] = 500.0
    code, values = cache[0].cpu(), cache[1].cpu()
    code[slots[0][3], 3] = -127  # against queries that are all positive
    q = torch.rand((1, 24, hq, 128), generator=g).add(0.5).to(dtype)
    ks[3] = 0.03
    cache[0].copy_(code)
    cache[2][slots[0].cuda(), 0, slots[1].cuda()] = ks.cuda()
    cache[3][slots[0].cuda(), 0, slots[1].cuda()] = vs.cuda()
    k = code[slots].reshape(1, 700, 1, 128).double() * ks.double()[None, :, None, None]
    v = values[slots].reshape(1, 700, 1, 128).double() * vs.double()[None, :, None, None]
    tree = torch.full((1, 24), 1, dtype=torch.int64)
    tree[0] |= torch.tensor([1 << t for t in range(24)])
    o, lse = outputs(c)
    S.spmm_execute_attn_cache8(plan(S, c), q.cuda(), *cache, o, lse, table=table.cuda(), tree=tree.cuda(), starts=ints([676]))
    want = R.attention(c, q.double(), k, v, A.sees(c, None, [700], [676], tree))
    A.check("o", o, *want["o"])
    A.check("lse", lse, *want["lse"])


@pytest.mark.parametrize("nq", [1, 24])
def test_cache8_values_of_zero(S, nq):
    """Zero scales, as rows of zeros have them: outputs of zero, and lse as it is."""
    c = case(nq=nq, nk=300, hq=8, hk=2, d=64, dtype=HF)
    g = torch.Generator().manual_seed(34)
    cache, k, v, table = filled(S, c, g)
    cache[3].zero_()
    q = torch.randn((1, nq, 8, 64), generator=g).to(HF)
    o, lse = outputs(c)
    S.spmm_execute_attn_cache8(plan(S, c), q.cuda(), *cache, o, lse, table=table.cuda(), starts=ints([300 - nq]))
    assert (o == 0).all()
    A.check("lse", lse, *R.attention(c, q.double(), k, 0 * v, A.sees(c, None, [300], [300 - nq], None))["lse"])


# and 33 to 64 rows of a list in both types, in ranges and whole
WEIGHTS = CACHE + [case(nq=24, nk=777, hq=8, hk=4, dtype=HF), case(b=2, nq=24, nk=900, hq=4, hk=2, d=128, dtype=HF),
                   case(b=3, nq=17, nk=4000, hq=3, hk=1, d=128), case(b=2, nq=150, nk=300, hq=4, hk=2, dtype=HF)]


def contiguous(cache, table, nk):
    """The same cache without a table: [b, nk, hk, d] and [b * nkb, hk, 64]."""
    at = table.long().cuda()
    return [x[at].flatten(1, 2)[:, :nk].contiguous() for x in cache[:2]] + [x[at].flatten(0, 1).contiguous() for x in cache[2:]]


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("how", ["full", "ragged"])
@pytest.mark.parametrize("n", range(len(WEIGHTS)))
def test_cache8_rounds_the_output_alone(S, n, how, paged):
    """Weights keep 16 bits in every kernel: what is left is the output's own rounding."""
    c = WEIGHTS[n]
    g = torch.Generator().manual_seed(650 + n)
    cache, k, v, table = filled(S, c, g)
    q = torch.randn((c["b"], c["nq"], c["hq"], c["d"]), generator=g).to(c["dtype"])
    lens, starts = new_tokens(c, how)
    o, lse = outputs(c)
    S.spmm_execute_attn_cache8(plan(S, c), q.cuda(), *(cache if paged else contiguous(cache, table, c["nk"])), o, lse,
                               table=table.cuda() if paged else None, lens=ints(lens), starts=ints(starts))
    want = R.attention8(c, q.double(), k, v, A.sees(c, None, lens, starts, None))
    A.check("o", o, *want["o"])
    A.check("lse", lse, *want["lse"])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hq", [1, 2, 4, 12])
@pytest.mark.parametrize("large", [(3,), (40,), (699,), (3, 699), (40, 675, 699)])
def test_cache8_large_values_leave_the_others(S, dtype, hq, large):
    """Values near f16's end, 2^27 times the others: at keys whose weight is about
    2^-60, and at a drafted token that only the last row sees.  The other rows
    keep all digits of their type: values of one sign, so that no output is small
    against them, and bounds in which a large value counts by its weight."""
    c = case(nq=24, nk=700, hq=hq, hk=1, d=128, dtype=dtype)
    g = torch.Generator().manual_seed(35)
    cache, _, _, table = filled(S, c, g)
    at = table.long()[0]
    slots = at.repeat_interleave(PAGE)[:700], torch.arange(700) % PAGE
    ks, vs = torch.full((700,), 1 / 700.0), torch.full((700,), 500.0 * 2.0 ** -27)
    code = cache[0].cpu()
    values = torch.randint(60, 128, cache[1].shape, generator=g).to(torch.int8)
    for j in large:
        vs[j] = 500.0
        if j < 676:  # against queries that are all positive
            code[slots[0][j], j % PAGE] = -127
            ks[j] = 0.03
    q = torch.rand((1, 24, hq, 128), generator=g).add(0.5).to(dtype)
    cache[0].copy_(code)
    cache[1].copy_(values)
    cache[2][slots[0].cuda(), 0, slots[1].cuda()] = ks.cuda()
    cache[3][slots[0].cuda(), 0, slots[1].cuda()] = vs.cuda()
    k = code[slots].reshape(1, 700, 1, 128).double() * ks.double()[None, :, None, None]
    v = values[slots].reshape(1, 700, 1, 128).double() * vs.double()[None, :, None, None]
    tree = torch.full((1, 24), 1, dtype=torch.int64)
    tree[0] |= torch.tensor([1 << t for t in range(24)])
    o, lse = outputs(c)
    S.spmm_execute_attn_cache8(plan(S, c), q.cuda(), *cache, o, lse, table=table.cuda(), tree=tree.cuda(), starts=ints([676]))
    want = R.attention8(c, q.double(), k, v, A.sees(c, None, [700], [676], tree))
    A.check("o", o, *want["o"])
    A.check("lse", lse, *want["lse"])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("nq,hq,nk", [(1, 4, 4097), (1, 1, 1), (24, 1, 300), (3, 4, 65), (24, 2, 900), (24, 4, 900), (24, 12, 700)])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("scale", [math.nan, math.inf])
def test_cache8_keys_and_values_that_stand_for_nan(S, dtype, nq, hq, nk, what, scale):
    """A row of codes 0 with a scale that is NaN or infinite, at a key that every
    query sees, at the first key of the last block, or at one that the last query
    alone sees: whoever sees it comes out as NaN, whoever does not as NaN or right
    (its block may spread it), and no score or sum of another row takes part."""
    c = case(nq=nq, nk=nk, hq=hq, hk=1, d=128, dtype=dtype)
    for at in sorted({0, nk // 2, (nk - nq) // PAGE * PAGE, nk - 1}):
        g = torch.Generator().manual_seed(36)
        cache, k, v, table = filled(S, c, g)
        q = torch.randn((1, nq, hq, 128), generator=g).to(dtype)
        want = R.attention8(c, q.double(), k, v, A.sees(c, None, [nk], [nk - nq], None))
        slot = int(table[0, at // PAGE])
        code, x = (cache[0], cache[2]) if what == "k" else (cache[1], cache[3])
        code[slot, at % PAGE], x[slot, :, at % PAGE] = 0, scale
        o, lse = outputs(c)
        S.spmm_execute_attn_cache8(plan(S, c), q.cuda(), *cache, o, lse, table=table.cuda(), starts=ints([nk - nq]))
        o, lse = o.cpu().double()[0], lse.cpu().double()[0].transpose(0, 1)  # [nq, hq, ..]
        sees = torch.arange(nk - nq, nk) >= at
        value, bound = want["o"][0][0], want["o"][1][0]
        assert o[sees].isnan().all(), at
        assert (o[~sees].isnan() | ((o - value).abs() <= bound)[~sees]).all(), at
        exact, off = (x[0].transpose(0, 1) for x in want["lse"])
        kept = torch.ones(nq, dtype=torch.bool) if what == "v" else ~sees
        assert lse[~kept].isnan().all() and ((lse - exact).abs() <= off)[kept].all(), at


def test_cache8_far_pages_and_strides(S):
    """Pages beyond 4 GiB of codes, k and v side by side in a page, heads first."""
    c = case(b=2, nq=2, nk=300, hq=8, hk=2, d=128)
    g = torch.Generator().manual_seed(32)
    pages = 70000
    base, k, v, table = filled(S, c, g)
    far = torch.randperm(pages - 60000, generator=g)[:10].reshape(2, 5).int() + 60000
    both = torch.empty((pages, 2, 2, PAGE, 256), dtype=torch.int8, device="cuda")  # [page][k, v][head][token][2 d]: 4.6 GB
    k8, v8 = (both[:, i, :, :, 64:192].transpose(1, 2) for i in range(2))
    ks, vs = torch.empty((2, pages, 2, PAGE), device="cuda")
    at, to = table.long().cuda().flatten(), far.long().cuda().flatten()
    for dst, src in zip((k8, v8, ks, vs), base):
        dst[to] = src[at]
    q = torch.randn((2, 2, 8, 128), generator=g).to(BF)
    P = plan(S, c)
    outs = []
    for cache, tab in ((base, table), ((k8, v8, ks, vs), far)):
        o, lse = outputs(c)
        S.spmm_execute_attn_cache8(P, q.cuda(), *cache, o, lse, table=tab.cuda(), starts=ints([298, 250]))
        kr, vr = torch.zeros((2, 2, 300, 2, 128), dtype=BF, device="cuda")
        S.spmm_execute_attn_read(P, *cache, kr, vr, table=tab.cuda())
        x = torch.randn((2, 2, 2, 128), generator=torch.Generator().manual_seed(1)).to(BF).cuda()
        S.spmm_execute_attn_write(P, x, x, *cache, table=tab.cuda(), starts=ints([298, 250]))
        o2, lse2 = outputs(c)
        S.spmm_execute_attn_cache8(P, q.cuda(), *cache, o2, lse2, table=tab.cuda(), starts=ints([298, 250]))
        outs.append((o, lse, kr, vr, o2, lse2))
    assert all(torch.equal(x, y) for x, y in zip(*outs)) and not torch.equal(outs[0][0], outs[0][4])
    want = R.attention(c, q.double(), k, v, A.sees(c, None, [300, 300], [298, 250], None))
    A.check("o", outs[1][0], *want["o"])


# ---- a run of them together ------------------------------------------------

def test_a_step_in_a_graph(S):
    """Decode steps captured once: norm and rotation, write, pool, choice of blocks,
    attention; every replay with new inputs is the eager calls' result, and
    the plain form's."""
    b, hq, hk, d, room, blocks = 3, 8, 2, 128, 640, 4
    nkb = room // PAGE
    g = torch.Generator().manual_seed(41)
    rope = S.spmm_plan_attn_rope(b, 1, hq, hk, d, R.freqs(64))
    P = S.spmm_plan_attn(b, 1, room, hq, hk, d, max_blocks=blocks)
    w = (1 + 0.1 * torch.randn((2, d), generator=g)).cuda()
    table = torch.randperm(b * nkb, generator=g).reshape(b, nkb).int().cuda()
    qkv = torch.empty((b, 1, hq + 2 * hk, d), dtype=BF, device="cuda")
    lens, starts = torch.zeros((2, b), dtype=torch.int32, device="cuda")

    def state():
        return (*empty_cache(b * nkb, hk, d), torch.zeros((b * nkb, hk, d), dtype=torch.int8, device="cuda"),
                torch.zeros((b * nkb, hk), device="cuda"), torch.empty((b, hk, 1, blocks), dtype=torch.int32, device="cuda"),
                torch.empty((b, 1, hq, d), dtype=BF, device="cuda"), torch.empty((b, 1, hk, d), dtype=BF, device="cuda"),
                torch.empty((b, 1, hq, d), dtype=BF, device="cuda"), torch.empty((b, hq, 1), device="cuda"))

    def step(s):
        k8, v8, ks, vs, pooled, scale, lists, q, k, o, lse = s
        x, y, v = qkv.split((hq, hk, hk), 2)
        S.spmm_execute_attn_rope(rope, x, y, q, k, q_weight=w[0], k_weight=w[1], lens=lens, starts=starts)
        S.spmm_execute_attn_write(P, k, v, k8, v8, ks, vs, table=table, lens=lens, starts=starts)
        S.spmm_execute_attn_pool8(P, k8, ks, pooled, scale, lens=lens, table=table, first=starts)
        S.spmm_execute_attn_select(P, q, pooled, scale, lists, lens=lens, starts=starts, table=table)
        S.spmm_execute_attn_cache8(P, q, k8, v8, ks, vs, o, lse, table=table, lists=lists, lens=lens, starts=starts)

    eager, kept = state(), state()
    side = torch.cuda.Stream()
    qkv.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(kept)
    at = [0, 130, 62]
    for s in (eager, kept):  # the texts so far
        gg = torch.Generator().manual_seed(42)
        for i in range(2):
            code, scale = R.encode(torch.randn((b * nkb, PAGE, hk, d), generator=gg).to(BF))
            s[i].copy_(code)
            s[2 + i].copy_(scale.transpose(1, 2))
        full = torch.tensor(at, dtype=torch.int32, device="cuda")
        Pf = S.spmm_plan_attn(b, room, room, hq, hk, d)
        S.spmm_execute_attn_pool8(Pf, s[0], s[2], s[4], s[5], lens=full, table=table, first=torch.zeros_like(full))
    for n in range(70):
        qkv.copy_(torch.randn(qkv.shape, generator=g).to(BF))
        starts.copy_(torch.tensor([a + n for a in at], dtype=torch.int32))
        lens.copy_(starts + 1)
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(eager, kept):
            assert torch.equal(torch.nan_to_num(x.float()), torch.nan_to_num(y.float())), n
    c = case(b=b, nq=1, nk=room, hq=hq, hk=hk, d=d, blocks=blocks)
    k8, v8, ks, vs, _, _, lists, q, _, o, lse = [x.cpu() for x in eager]
    page = table.long().cpu()
    k, v = (torch.nan_to_num(R.values(code, scale)[page]).flatten(1, 2) for code, scale in ((k8, ks), (v8, vs)))
    want = R.attention(c, q.double(), k, v, A.sees(c, lists, lens.tolist(), starts.tolist(), None))
    A.check("o", o, *want["o"])
    A.check("lse", lse, *want["lse"])


def test_training_step_with_rotation(S):
    """Norm and rotation, attention over lists, and both gradients chained: against
    autograd of the whole in 64 bits, within what bf16 between the calls leaves
    (each of q, k, o, their gradients and P is rounded once, 2^-8 of itself: the
    norm of the difference stays below eight such steps of the result's)."""
    b, n, hq, hk, d = 2, 200, 4, 2, 64
    g = torch.Generator().manual_seed(51)
    q, k, v, grad = (torch.randn((b, n, h, d), generator=g).to(BF) for h in (hq, hk, hk, hq))
    w = 1 + 0.2 * torch.randn((2, d), generator=g)
    rope = S.spmm_plan_attn_rope(b, n, hq, hk, d, R.freqs(32), backward=True)
    P = S.spmm_plan_attn(b, n, n, hq, hk, d, max_blocks=4, backward=True)
    lists = torch.arange(4, dtype=torch.int32).expand(b, hk, 4, 4).contiguous().cuda()
    qg, kg, vg, gg, wg = (x.cuda() for x in (q, k, v, grad, w))
    qo, ko, o, lse = torch.empty_like(qg), torch.empty_like(kg), torch.empty_like(qg), torch.empty((b, hq, n), device="cuda")
    S.spmm_execute_attn_rope(rope, qg, kg, qo, ko, q_weight=wg[0], k_weight=wg[1])
    S.spmm_execute_attn(P, qo, ko, vg, lists, o, lse)
    dqo, dko, dv = torch.empty_like(qg), torch.empty_like(kg), torch.empty_like(vg)
    S.spmm_execute_attn_backward(P, gg, qo, ko, vg, lists, o, lse, dqo, dko, dv)
    dw = torch.empty((2, d), device="cuda")
    S.spmm_execute_attn_rope_backward(rope, dqo, dko, qg, kg, dqo, dko, q_weight=wg[0], k_weight=wg[1],
                                      dq_weight=dw[0], dk_weight=dw[1])
    leaves = [x.double().requires_grad_() for x in (q, k, v, w[0], w[1])]
    angle, _ = R.angles(R.freqs(32), [0] * 32, torch.arange(n).expand(1, b, n))

    def turned(x, w):
        y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        return R.turn(y, torch.cos(angle), torch.sin(angle), False)

    qt, kt = turned(leaves[0], leaves[3]).transpose(1, 2), turned(leaves[1], leaves[4]).transpose(1, 2).repeat_interleave(2, 1)
    s = (qt @ kt.transpose(-1, -2) / math.sqrt(d)).masked_fill(~torch.ones(n, n, dtype=torch.bool).tril(), -math.inf)
    want = (torch.softmax(s, -1) @ leaves[2].transpose(1, 2).repeat_interleave(2, 1)).transpose(1, 2)
    found = torch.autograd.grad(want, leaves, grad.double())
    for name, x, y in zip(("o", "dq", "dk", "dv", "dqw", "dkw"), (o, dqo, dko, dv, dw[0], dw[1]), (want.detach(), *found)):
        off = ((x.cpu().double() - y).norm() / y.norm()).item()
        print(f"{name}: off by {off:.1e} of the norm", flush=True)
        assert off < 8 * 2.0 ** -8, name


def test_two_plans_on_two_streams(S):
    """Calls of the same kind at once, each with a plan of its own."""
    c = case(b=2, nq=1, nk=5000, hq=8, hk=2, d=128)
    g = torch.Generator().manual_seed(61)
    cache, _, _, table = filled(S, c, g)
    q = torch.randn((2, 1, 8, 128), generator=g).to(BF).cuda()
    rc = rope_case(b=2, n=500, hq=8, hk=2, d=128)
    x, y, gx, gy, qw, kw, *_ = rope_inputs(rc, 62)
    x, y, gx, gy, qw, kw = (t.cuda() for t in (x, y, gx, gy, qw, kw))
    tab, starts = table.cuda(), ints([4999, 4999])

    def work(P, Q, s):
        o, lse = outputs(c)
        dx, dy, dw = torch.empty_like(x), torch.empty_like(y), torch.empty((2, 128), device="cuda")
        for _ in range(3):
            S.spmm_execute_attn_cache8(P, q, *cache, o, lse, table=tab, starts=starts, stream=s)
            S.spmm_execute_attn_rope_backward(Q, gx, gy, x, y, dx, dy, q_weight=qw, k_weight=kw, dq_weight=dw[0],
                                              dk_weight=dw[1], stream=s)
        return o, lse, dx, dy, dw

    alone = work(plan(S, c), rope_plan(S, rc, backward=True), torch.cuda.current_stream())
    torch.cuda.synchronize()
    plans = [(plan(S, c), rope_plan(S, rc, backward=True), torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    outs = [work(*p) for p in plans]
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(alone, got))


def test_plans_from_numpy_sizes(S):
    """Sizes and a device that are numpy's whole numbers plan for the same tensors."""
    i = np.int64
    q, k = torch.ones((1, 2, 2, 64), dtype=BF, device="cuda"), torch.ones((1, 2, 1, 64), dtype=BF, device="cuda")
    R1 = S.spmm_plan_attn_rope(i(1), i(2), i(2), i(1), i(64), R.freqs(32), axes=i(1), device=i(0))
    S.spmm_execute_attn_rope(R1, q, k, q, k, q_weight=torch.ones(64, device="cuda"))
    P = S.spmm_plan_attn(i(1), i(2), i(64), i(2), i(1), i(64), device=i(0))
    k8, v8, ks, vs = empty_cache(1, 1, 64)
    S.spmm_execute_attn_write(P, k, k, k8, v8, ks, vs, table=ints([[0]]))
    o, lse = torch.empty_like(q), torch.empty((1, 2, 2), device="cuda")
    S.spmm_execute_attn_cache8(P, q, k8, v8, ks, vs, o, lse, table=ints([[0]]), lens=ints([2]))
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


def test_calls_without_the_module(S, monkeypatch):
    """The same results and refusals where the tensors are checked in Python."""
    c = case(b=2, nq=1, nk=300, hq=8, hk=2, d=128)
    g = torch.Generator().manual_seed(63)
    cache, _, _, table = filled(S, c, g)
    q = torch.randn((2, 1, 8, 128), generator=g).to(BF).cuda()
    outs = []
    for checks in (S._load_binding(), S._PythonChecks):
        monkeypatch.setattr(S, "_bind", checks)
        o, lse = outputs(c)
        S.spmm_execute_attn_cache8(plan(S, c), q, *cache, o, lse, table=table.cuda(), starts=ints([299, 100]))
        outs.append((o, lse))
        test_binding_refuses_tensors(S)
    assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_binding_refuses_tensors(S):
    P = S.spmm_plan_attn(1, 1, 64, 2, 1, 64)
    Q = S.spmm_plan_attn_rope(1, 1, 2, 1, 64, R.freqs(32))
    k8, v8, ks, vs = empty_cache(1, 1, 64)
    q, k = torch.zeros((1, 1, 2, 64), dtype=BF, device="cuda"), torch.zeros((1, 1, 1, 64), dtype=BF, device="cuda")
    table = ints([[0]])
    o, lse = torch.empty_like(q), torch.empty((1, 2, 1), device="cuda")
    for bad in (lambda: S.spmm_execute_attn_cache8(P, q, k8.short(), v8, ks, vs, o, lse, table=table),
                lambda: S.spmm_execute_attn_cache8(P, q, k8, v8, ks[:, :, :32], vs, o, lse, table=table),
                lambda: S.spmm_execute_attn_cache8(P, q, k8, v8.cpu(), ks, vs, o, lse, table=table),
                lambda: S.spmm_execute_attn_cache8(Q, q, k8, v8, ks, vs, o, lse, table=table),
                lambda: S.spmm_execute_attn_write(P, k.half(), k, k8, v8, ks, vs, table=table),
                lambda: S.spmm_execute_attn_write(P, k, k, k8, v8, ks.double(), vs, table=table),
                lambda: S.spmm_execute_attn_rope(P, q, k, q, k),
                lambda: S.spmm_execute_attn_rope(Q, q, k, q, k, q_weight=torch.ones(63, device="cuda")),
                lambda: S.spmm_execute_attn_rope(Q, q, k, q, k, positions=ints([[0]]))):
        with pytest.raises(ValueError):
            bad()
