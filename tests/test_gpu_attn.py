"""Block-sparse attention on the GPU against the plain 64-bit form
(attn_ref.py), whose bounds count the roundings of each output."""
import math

import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module")
def S():
    import sparse_dense_matrix_amd as S
    assert torch.cuda.is_available()
    return S


def case(b=1, nq=64, nk=None, hq=4, hk=2, d=64, dtype=torch.bfloat16, q_block=64, blocks=4, **kw):
    return dict(b=b, nq=nq, nk=nq if nk is None else nk, hq=hq, hk=hk, d=d, dtype=dtype, q_block=q_block,
                blocks=blocks, **kw)


def code(S, c):
    return S.BF16 if c["dtype"] == torch.bfloat16 else S.F16


def plan(S, c, **kw):
    return S.spmm_plan_attn(c["b"], c["nq"], c["nk"], c["hq"], c["hk"], c["d"], dtype=code(S, c),
                            q_block=c["q_block"], max_blocks=c["blocks"], scale=c.get("scale"), **kw)


def inputs(c, seed):
    g = torch.Generator().manual_seed(seed)

    def make(*shape):
        return torch.randn(shape, generator=g).to(c["dtype"])

    return (make(c["b"], c["nq"], c["hq"], c["d"]), make(c["b"], c["nk"], c["hk"], c["d"]),
            make(c["b"], c["nk"], c["hk"], c["d"]), make(c["b"], c["nq"], c["hq"], c["d"]), g)


def random_lists(c, g, empty=0.0):
    """Ascending blocks of the whole sequence, some lists short or empty."""
    nkb, nqb = -(-c["nk"] // PAGE), -(-c["nq"] // c["q_block"])
    lists = torch.full((c["b"], c["hk"], nqb, c["blocks"]), -1, dtype=torch.int32)
    for x in lists.reshape(-1, c["blocks"]):
        n = 0 if torch.rand(1, generator=g) < empty else int(torch.randint(1, min(nkb, c["blocks"]) + 1, (1,), generator=g))
        x[:n] = torch.randperm(nkb, generator=g)[:n].sort().values.int()
    return lists


def poison(x):
    return torch.full_like(x, float("nan"))


def dev(x):
    return None if x is None else x.cuda()


def run_forward(S, c, q, k, v, lists, lens, starts, P=None, stream=None):
    P = P or plan(S, c)
    o = torch.full((c["b"], c["nq"], c["hq"], c["d"]), float("nan"), dtype=c["dtype"], device="cuda")
    lse = torch.full((c["b"], c["hq"], c["nq"]), float("nan"), device="cuda")
    S.spmm_execute_attn(P, q, k, v, lists, o, lse, lens=lens, starts=starts, stream=stream)
    return o, lse


FORWARD = [
    case(nq=1, nk=1, blocks=1), case(nq=1, nk=65, hq=8, hk=1, d=128), case(nq=63, hq=3, hk=3, q_block=16),
    case(b=2, nq=130, hq=6, hk=2, q_block=16, dtype=torch.float16), case(nq=200, d=128, hq=8, hk=2),
    case(nq=129, hq=16, hk=1, q_block=1, blocks=2, d=128), case(nq=40, nk=300, hq=5, hk=1, q_block=4, blocks=5),
    case(b=3, nq=70, nk=257, hq=8, hk=8, q_block=32, blocks=3, d=128, dtype=torch.float16),
    case(nq=64, nk=640, hq=10, hk=2, blocks=10, d=128, scale=0.3), case(nq=257, hq=4, hk=4, q_block=64, blocks=70),
    case(nq=96, nk=4800, hq=2, hk=1, blocks=75, q_block=32),
]


def lengths(c, g, kind):
    b, nq, nk = c["b"], c["nq"], c["nk"]
    if kind == "full":
        lens, starts = [nk] * b, [nk - nq] * b
    elif kind == "ragged":
        lens = [int(torch.randint(1, nk + 1, (1,), generator=g)) for _ in range(b)]
        starts = [max(0, n - nq) for n in lens]
    else:  # rows before the first key and past the last, empty sequences, odd values
        lens = [[0, nk // 2, nk + 7][(i + 1) % 3] for i in range(b)]
        starts = [[-3, nk // 2 - nq // 2, -(2 ** 31)][i % 3] for i in range(b)]
    return torch.tensor(lens, dtype=torch.int32), torch.tensor(starts, dtype=torch.int32)


@pytest.mark.parametrize("kind", ["full", "ragged", "odd"])
@pytest.mark.parametrize("n", range(len(FORWARD)))
def test_forward(S, n, kind):
    c = FORWARD[n]
    q, k, v, _, g = inputs(c, 100 + n)
    lens, starts = lengths(c, g, kind)
    lists = random_lists(c, g, empty=0.2)
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), lens.cuda(), starts.cuda())
    w = R.sees(c, lists, lens, starts, None)
    want = R.attention(c, q.double(), k.double(), v.double(), w)
    R.check("o", o, *want["o"])
    R.check("lse", lse, *want["lse"])


def test_forward_without_lens(S):
    c = case(nq=100, blocks=2)
    q, k, v, _, g = inputs(c, 7)
    lists = random_lists(c, g)
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), None, None)
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, lists, [100], [0], None))
    R.check("o", o, *want["o"])
    R.check("lse", lse, *want["lse"])


def test_forward_list_entries_that_read_nothing(S):
    """Ids out of range, gaps of -1, a block named twice."""
    c = case(nq=64, nk=256, hq=2, hk=1, blocks=6)
    q, k, v, _, g = inputs(c, 8)
    lists = torch.tensor([-1, 1, 1, -7, 2 ** 31 - 1, 4], dtype=torch.int32).reshape(1, 1, 1, 6)
    starts, lens = torch.tensor([150], dtype=torch.int32), torch.tensor([214], dtype=torch.int32)
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), lens.cuda(), starts.cuda())
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, lists, lens, starts, None))
    R.check("o", o, *want["o"])
    R.check("lse", lse, *want["lse"])


def test_forward_ignores_what_stands_past_the_length(S):
    c = case(b=2, nq=90, hq=4, hk=2, blocks=2, d=128)
    q, k, v, _, g = inputs(c, 9)
    lens, starts = torch.tensor([70, 1], dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    k[0, 70:], v[0, 70:], k[1, 1:], v[1, 1:] = float("nan"), float("inf"), float("inf"), float("nan")
    q[0, 70:], q[1, 1:] = float("nan"), float("inf")
    lists = torch.tensor([0, 1], dtype=torch.int32).expand(2, 2, 2, 2).contiguous()
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), lens.cuda(), starts.cuda())
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, lists, lens, starts, None))
    R.check("o", o, *want["o"])
    R.check("lse", lse, *want["lse"])


def test_forward_scores_far_apart(S):
    """Scores over hundreds: the maximum moves, weights underflow to zero."""
    c = case(nq=64, nk=512, hq=2, hk=1, blocks=8, d=64)
    q, k, v, _, g = inputs(c, 10)
    k = (k.float() * torch.linspace(0.1, 40, 512)[None, :, None, None]).to(c["dtype"])
    lists = torch.arange(8, dtype=torch.int32).reshape(1, 1, 1, 8)
    starts = torch.tensor([448], dtype=torch.int32)
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), None, starts.cuda())
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, lists, [512], starts, None))
    R.check("o", o, *want["o"])
    R.check("lse", lse, *want["lse"])


def strided(x, how):
    """The same values with other strides."""
    if how == "heads first":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if how == "padded":
        wide = torch.zeros((*x.shape[:2], x.shape[2] + 1, x.shape[3] + 8), dtype=x.dtype, device=x.device)
        wide[:, :, 1:, 8:] = x
        return wide[:, :, 1:, 8:]
    wide = torch.zeros((x.shape[0], x.shape[1], 3, *x.shape[2:]), dtype=x.dtype, device=x.device)
    wide[:, :, 1] = x
    return wide[:, :, 1]


@pytest.mark.parametrize("how", ["heads first", "padded", "packed"])
def test_forward_backward_strides(S, how):
    c = case(b=2, nq=100, hq=6, hk=2, q_block=16, blocks=2, d=64)
    q, k, v, grad, g = inputs(c, 11)
    lists = random_lists(c, g, empty=0.1)
    base = [t.cuda() for t in (q, k, v, grad)]
    other = [strided(t, how) for t in base]
    outs = []
    for q1, k1, v1, g1 in (base, other):
        P = plan(S, c, backward=True)
        o, lse = strided(torch.zeros_like(base[0]), how), torch.zeros((2, 6, 100), device="cuda")
        if q1 is base[0]:
            o = o.contiguous()
        S.spmm_execute_attn(P, q1, k1, v1, lists.cuda(), o, lse)
        dq, dk, dv = torch.empty_like(q1), torch.empty_like(k1), torch.empty_like(v1)
        S.spmm_execute_attn_backward(P, g1, q1, k1, v1, lists.cuda(), o, lse, dq, dk, dv)
        outs.append([t.clone().contiguous() for t in (o, lse, dq, dk, dv)])
    for x, y in zip(*outs):
        assert torch.equal(x, y)


def test_forward_broadcast_heads(S):
    c = case(nq=80, hq=4, hk=4, blocks=2)
    q, k, v, _, g = inputs(c, 12)
    k, v = k[:, :, :1], v[:, :, :1]
    lists = random_lists(c, g)
    o, lse = run_forward(S, c, q.cuda(), k.cuda().expand(-1, -1, 4, -1), v.cuda().expand(-1, -1, 4, -1),
                         lists.cuda(), None, None)
    o2, lse2 = run_forward(S, c, q.cuda(), k.cuda().repeat(1, 1, 4, 1), v.cuda().repeat(1, 1, 4, 1),
                           lists.cuda(), None, None)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


BACKWARD = [
    case(nq=1, nk=1, blocks=1), case(nq=63, hq=3, hk=3, q_block=16, blocks=1),
    case(b=2, nq=130, hq=6, hk=2, q_block=16), case(nq=200, d=128, hq=8, hk=2),
    case(nq=129, hq=16, hk=1, q_block=1, blocks=2, d=128), case(nq=40, nk=300, hq=5, hk=1, q_block=4, blocks=5),
    case(b=3, nq=70, nk=257, hq=8, hk=8, q_block=32, blocks=3, d=128, dtype=torch.float16),
    case(nq=64, nk=640, hq=10, hk=2, blocks=10, d=128, scale=0.3), case(nq=700, hq=1, hk=1, q_block=1, blocks=3),
    case(nq=700, hq=2, hk=1, q_block=64, blocks=3, d=128),
]


@pytest.mark.parametrize("kind", ["full", "ragged", "odd"])
@pytest.mark.parametrize("n", range(len(BACKWARD)))
def test_backward(S, n, kind):
    c = BACKWARD[n]
    q, k, v, grad, g = inputs(c, 200 + n)
    lens, starts = lengths(c, g, kind)
    lists = random_lists(c, g, empty=0.2)
    for i in range(c["b"]):  # what no query or key uses may hold anything
        n_i = min(max(int(lens[i]), 0), c["nk"])
        k[i, n_i:], v[i, n_i:] = float("nan"), float("inf")
        for t in range(c["nq"]):
            if not 0 <= int(starts[i]) + t < n_i:
                q[i, t], grad[i, t] = float("nan"), float("inf")
    P = plan(S, c, backward=True)
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), lens.cuda(), starts.cuda(), P)
    dq, dk, dv = (torch.full_like(t, float("nan")).cuda() for t in (q, k, v))
    S.spmm_execute_attn_backward(P, grad.cuda(), q.cuda(), k.cuda(), v.cuda(), lists.cuda(), o, lse, dq, dk, dv,
                                 lens=lens.cuda(), starts=starts.cuda())
    w = R.sees(c, lists, lens, starts, None)
    want = R.attention(c, q.double(), k.double(), v.double(), w, grad.double())
    for name, got in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        R.check(name, got, *want[name])


def test_backward_long_inverse_list(S):
    """One block that every list names: its query blocks are cut into items."""
    c = case(nq=2600, hq=2, hk=2, q_block=1, blocks=2)
    q, k, v, grad, g = inputs(c, 30)
    nqb = c["nq"]
    lists = torch.zeros((1, 2, nqb, 2), dtype=torch.int32)
    lists[..., 1] = torch.arange(nqb, dtype=torch.int32) // PAGE
    lists[..., 1][lists[..., 1] == 0] = -1
    P = plan(S, c, backward=True)
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), None, None, P)
    outs = []
    for _ in range(2):
        dq, dk, dv = (torch.full_like(t, float("nan")).cuda() for t in (q, k, v))
        S.spmm_execute_attn_backward(P, grad.cuda(), q.cuda(), k.cuda(), v.cuda(), lists.cuda(), o, lse, dq, dk, dv)
        outs.append((dq, dk, dv))
    assert all(torch.equal(x, y) for x, y in zip(*outs)), "not the same bits twice"
    nkb = -(-c["nk"] // PAGE)
    key = torch.arange(c["nk"])
    t = torch.arange(c["nq"])
    w = ((key[None] <= t[:, None]) & ((key[None] // PAGE == 0) | (key[None] // PAGE == t[:, None] // PAGE)))
    w = w.double().expand(1, 2, -1, -1)
    assert nkb == 41
    want = R.attention(c, q.double(), k.double(), v.double(), w, grad.double())
    for name, got in (("o", o), ("lse", lse), ("dq", outs[0][0]), ("dk", outs[0][1]), ("dv", outs[0][2])):
        R.check(name, got, *want[name])


# ---- cache -----------------------------------------------------------------

def paged(c, k, v, g, spare=3):
    """Pages in an order of their own, NaN in the spare ones."""
    nkb = -(-c["nk"] // PAGE)
    pages = c["b"] * nkb + spare
    table = torch.randperm(pages, generator=g)[:c["b"] * nkb].reshape(c["b"], nkb).int()
    kp = torch.full((pages, PAGE, c["hk"], c["d"]), float("nan"), dtype=c["dtype"])
    vp = kp.clone()
    for x, xp in ((k, kp), (v, vp)):
        pad = torch.full((c["b"], nkb * PAGE, c["hk"], c["d"]), float("nan"), dtype=c["dtype"])
        pad[:, :c["nk"]] = x
        xp[table.long()] = pad.reshape(c["b"], nkb, PAGE, c["hk"], c["d"])
    return kp, vp, table


CACHE = [
    case(nq=1, nk=64, blocks=2), case(b=3, nq=1, nk=640, hq=8, hk=2, d=128, blocks=3),
    case(b=2, nq=1, nk=5000 // 64 * 64, hq=4, hk=1, blocks=9), case(b=2, nq=5, nk=448, hq=16, hk=2, d=128, blocks=4),
    case(b=4, nq=24, nk=384, hq=8, hk=2, d=128, blocks=4, dtype=torch.float16), case(nq=64, nk=1024, hq=16, hk=1, blocks=8),
    case(b=2, nq=13, nk=192, hq=3, hk=3, blocks=2), case(nq=150, nk=640, hq=4, hk=4, blocks=6, d=128),
]


def run_cache(S, c, q, kp, vp, **kw):
    o = torch.full((c["b"], c["nq"], c["hq"], c["d"]), float("nan"), dtype=c["dtype"], device="cuda")
    lse = torch.full((c["b"], c["hq"], c["nq"]), float("nan"), device="cuda")
    P = plan(S, c)
    S.spmm_execute_attn_cache(P, q.cuda(), kp.cuda(), vp.cuda(), o, lse, **{n: dev(x) for n, x in kw.items()})
    return o, lse


@pytest.mark.parametrize("kind", ["full", "ragged", "odd"])
@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("n", range(len(CACHE)))
def test_cache(S, n, listed, kind):
    c = CACHE[n]
    q, k, v, _, g = inputs(c, 300 + n)
    lens, starts = lengths(c, g, kind)
    kp, vp, table = paged(c, k, v, g)
    for i in range(c["b"]):  # a page's keys past the length
        n_i = min(max(int(lens[i]), 0), c["nk"])
        if n_i < c["nk"]:
            kp[table[i, n_i // PAGE].long(), n_i % PAGE:] = float("nan")
            vp[table[i, n_i // PAGE].long(), n_i % PAGE:] = float("inf")
    lists = random_lists(c, g, empty=0.1) if listed else None
    o, lse = run_cache(S, c, q, kp, vp, table=table, lists=lists, lens=lens, starts=starts)
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, lists, lens, starts, None))
    R.check("o", o, *want["o"])
    R.check("lse", lse, *want["lse"])


@pytest.mark.parametrize("nq,listed", [(2, False), (24, False), (64, True), (33, True)])
def test_cache_tree(S, nq, listed):
    c = case(b=3, nq=nq, nk=320, hq=4, hk=2, d=128, blocks=3)
    q, k, v, _, g = inputs(c, 400 + nq)
    lens = torch.tensor([nq, 320, 200], dtype=torch.int32)
    starts = lens - nq
    tree = torch.randint(-2 ** 63, 2 ** 63 - 1, (3, nq), generator=g)
    tree[0, 1] = 0  # no drafted token and no text: nothing is seen
    kp, vp, table = paged(c, k, v, g)
    lists = random_lists(c, g) if listed else None
    o, lse = run_cache(S, c, q, kp, vp, table=table, lists=lists, lens=lens, starts=starts, tree=tree)
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, lists, lens, starts, tree))
    R.check("o", o, *want["o"])
    R.check("lse", lse, *want["lse"])
    assert torch.isinf(lse[0, :, 1]).all() and (o[0, 1] == 0).all()


def test_cache_pages_out_of_range_read_nothing(S):
    c = case(b=1, nq=2, nk=640, hq=4, hk=2, d=64, blocks=4)
    q, k, v, _, g = inputs(c, 500)
    kp, vp, table = paged(c, k, v, g)
    table[0, 1], table[0, 4], table[0, 9] = -1, kp.shape[0], 2 ** 31 - 1
    ok = torch.ones((1, 10))
    ok[0, [1, 4, 9]] = 0
    starts, lens = torch.tensor([600], dtype=torch.int32), torch.tensor([602], dtype=torch.int32)
    o, lse = run_cache(S, c, q, kp, vp, table=table, lens=lens, starts=starts)
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, None, lens, starts, None, ok))
    R.check("o", o, *want["o"])
    R.check("lse", lse, *want["lse"])


def test_cache_without_pages(S):
    c = case(b=2, nq=3, nk=300, hq=8, hk=2, d=128, blocks=2)
    q, k, v, _, g = inputs(c, 501)
    lens, starts = torch.tensor([300, 129], dtype=torch.int32), torch.tensor([297, 126], dtype=torch.int32)
    o, lse = run_cache(S, c, q, k, v, lens=lens, starts=starts)
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, None, lens, starts, None))
    R.check("o", o, *want["o"])
    R.check("lse", lse, *want["lse"])


# ---- choice of blocks ------------------------------------------------------

SELECT = [
    case(nq=64, blocks=2), case(b=2, nq=700, hq=6, hk=2, q_block=16, blocks=4), case(nq=900, hq=4, hk=4, q_block=64, blocks=5, d=128),
    case(nq=400, hq=16, hk=1, q_block=1, blocks=3, d=128, dtype=torch.float16), case(b=3, nq=1, nk=4096, hq=8, hk=2, blocks=16, d=128),
    case(b=2, nq=9, nk=1000, hq=5, hk=1, blocks=7), case(nq=32, nk=40000, hq=2, hk=1, q_block=32, blocks=600),
]


@pytest.mark.parametrize("kind", ["full", "ragged", "odd"])
@pytest.mark.parametrize("n", range(len(SELECT)))
def test_pool_and_select(S, n, kind):
    c = SELECT[n]
    q, k, v, _, g = inputs(c, 600 + n)
    lens, starts = lengths(c, g, kind)
    nkb, nqb = -(-c["nk"] // PAGE), -(-c["nq"] // c["q_block"])
    values = torch.zeros((c["b"] * nkb, c["hk"], c["d"]), dtype=torch.int8, device="cuda")
    scale = torch.zeros((c["b"] * nkb, c["hk"]), device="cuda")
    sink, local = (1, 1) if n % 2 else (0, 2)
    P = plan(S, c, sink_blocks=sink, local_blocks=local)
    S.spmm_execute_attn_pool(P, k.cuda(), values, scale, lens=lens.cuda())
    rv, rs = R.pool(k, lens, c["nk"])
    assert torch.equal(values.cpu().reshape(rv.shape), rv)
    assert torch.equal(scale.cpu().reshape(rs.shape), rs)
    lists = torch.full((c["b"], c["hk"], nqb, c["blocks"]), -9, dtype=torch.int32, device="cuda")
    S.spmm_execute_attn_select(P, q.cuda(), values, scale, lists, lens=lens.cuda(), starts=starts.cuda())
    assert torch.equal(lists.cpu(), R.select(c, q, rv, rs, lens, starts, sink, local))


def test_pool_pages_from_first(S):
    """Only the blocks from `first` on are written; bad pages are not."""
    c = case(b=3, nq=3, nk=640, hq=4, hk=2, d=128, blocks=3)
    q, k, v, _, g = inputs(c, 700)
    kp, vp, table = paged(c, k, v, g)
    lens = torch.tensor([640, 66, 130], dtype=torch.int32)
    first = torch.tensor([600, 63, 127], dtype=torch.int32)
    table[2, 2] = kp.shape[0] + 5
    values = torch.full((kp.shape[0], 2, 128), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((kp.shape[0], 2), 99.0, device="cuda")
    P = plan(S, c)
    S.spmm_execute_attn_pool(P, kp.cuda(), values, scale, lens=lens.cuda(), table=table.cuda(), first=first.cuda())
    rv, rs = R.pool(k, lens, c["nk"])
    written = {int(table[0, 9]): (0, 9), int(table[1, 0]): (1, 0), int(table[1, 1]): (1, 1), int(table[2, 1]): (2, 1)}
    for p in range(kp.shape[0]):
        if p in written:
            assert torch.equal(values[p].cpu(), rv[written[p]]) and torch.equal(scale[p].cpu(), rs[written[p]])
        else:
            assert (values[p] == 99).all() and (scale[p] == 99).all()


def test_select_ties_and_bad_scores(S):
    """Equal scores go to the lower block; zeros, infinities, missing pages."""
    c = case(b=1, nq=1, nk=1280, hq=2, hk=1, d=64, blocks=6)
    q, k, v, _, g = inputs(c, 701)
    values = torch.zeros((20, 1, 64), dtype=torch.int8)
    values[[4, 9, 11, 15], 0, 3] = 5
    scale = torch.ones((20, 1))
    scale[11], scale[2] = float("inf"), float("nan")
    q = torch.zeros_like(q)
    q[..., 3] = 1.0
    table = torch.arange(20, dtype=torch.int32).reshape(1, 20)
    table[0, 4] = -1
    P = plan(S, c)
    lists = torch.zeros((1, 1, 1, 6), dtype=torch.int32, device="cuda")
    starts = torch.tensor([1279], dtype=torch.int32, device="cuda")
    S.spmm_execute_attn_select(P, q.cuda(), values.cuda(), scale.cuda(), lists, starts=starts, table=table.cuda())
    # 0 and 19 always; 11 (infinite), 9 and 15, then the lowest zero: 1
    assert lists.flatten().tolist() == [0, 1, 9, 11, 15, 19]
    q[..., 5] = float("inf")  # a sum that is not finite: values 0, all scores 0
    S.spmm_execute_attn_select(P, q.cuda(), values.cuda(), scale.cuda(), lists, starts=starts, table=table.cuda())
    assert lists.flatten().tolist() == [0, 1, 3, 5, 6, 19]


# ---- streams, graphs, refusals ---------------------------------------------

def test_another_stream_and_graph(S):
    c = case(b=2, nq=200, hq=4, hk=2, q_block=16, blocks=3, d=128)
    q, k, v, grad, g = inputs(c, 800)
    lists = random_lists(c, g).cuda()
    q, k, v, grad = (t.cuda() for t in (q, k, v, grad))
    P = plan(S, c, backward=True)
    o, lse = torch.zeros_like(q), torch.zeros((2, 4, 200), device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    values = torch.zeros((2 * 4, 2, 128), dtype=torch.int8, device="cuda")
    scale = torch.zeros((2 * 4, 2), device="cuda")
    chosen = torch.zeros_like(lists)
    outs = (o, lse, dq, dk, dv, values, scale, chosen)

    def step(st):
        S.spmm_execute_attn_pool(P, k, values, scale, stream=st)
        S.spmm_execute_attn_select(P, q, values, scale, chosen, stream=st)
        S.spmm_execute_attn(P, q, k, v, chosen, o, lse, stream=st)
        S.spmm_execute_attn_backward(P, grad, q, k, v, chosen, o, lse, dq, dk, dv, stream=st)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    torch.cuda.synchronize()
    eager = [t.clone() for t in outs]
    assert all(t.float().abs().sum() > 0 for t in eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(torch.cuda.current_stream())
    for rep in range(3):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs, eager):
            assert torch.equal(x, y), f"replay {rep}"


def test_graph_cache_split(S):
    c = case(b=1, nq=1, nk=4096, hq=8, hk=2, d=128, blocks=4)
    q, k, v, _, g = inputs(c, 801)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    P = plan(S, c)
    assert P.info()["workspace_bytes"] > 0, "the case must cut the sequence into ranges"
    o, lse = torch.zeros_like(q), torch.zeros((1, 8, 1), device="cuda")
    starts = torch.tensor([4095], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    S.spmm_execute_attn_cache(P, q, k, v, o, lse, starts=starts, stream=s)
    torch.cuda.synchronize()
    eager = (o.clone(), lse.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        S.spmm_execute_attn_cache(P, q, k, v, o, lse, starts=starts, stream=torch.cuda.current_stream())
    for rep in range(3):
        o.zero_(), lse.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager[0]) and torch.equal(lse, eager[1])


def test_empty_shapes(S):
    for c in (case(b=0, nq=4, nk=64), case(nq=0, nk=64), case(nq=4, nk=0)):
        P = plan(S, c, backward=True)
        q, k, v, grad, _ = inputs(c, 1)
        q, k, v, grad = (t.cuda() for t in (q, k, v, grad))
        nqb = -(-c["nq"] // 64)
        lists = torch.zeros((c["b"], 2, nqb, 4), dtype=torch.int32, device="cuda")
        o, lse = torch.full_like(q, 9), torch.full((c["b"], 4, c["nq"]), 9.0, device="cuda")
        S.spmm_execute_attn(P, q, k, v, lists, o, lse)
        dq, dk, dv = torch.full_like(q, 9), torch.full_like(k, 9), torch.full_like(v, 9)
        S.spmm_execute_attn_backward(P, grad, q, k, v, lists, o, lse, dq, dk, dv)
        torch.cuda.synchronize()
        for t in (o, dq, dk, dv):
            assert (t == 0).all()
        assert (lse == -math.inf).all()


def test_refusals_of_tensors(S):
    c = case(nq=8, nk=64)
    P = plan(S, c)
    q, k, v, grad, g = inputs(c, 2)
    q, k, v, grad = (t.cuda() for t in (q, k, v, grad))
    lists = torch.zeros((1, 2, 1, 4), dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((1, 4, 8), device="cuda")
    for bad in (dict(q=q.half()), dict(q=q[:, :7]), dict(k=k.cpu()), dict(lists=lists.long()), dict(lse=lse[:, :3]),
                dict(v=v.transpose(2, 3).contiguous().transpose(2, 3)), dict(o=o.float())):
        a = dict(q=q, k=k, v=v, lists=lists, o=o, lse=lse)
        a.update(bad)
        with pytest.raises(ValueError):
            S.spmm_execute_attn(P, *a.values())
    with pytest.raises(S.SpmmError) as e:  # made without backward
        S.spmm_execute_attn_backward(P, grad, q, k, v, lists, o, lse, q.clone(), k.clone(), v.clone())
    assert e.value.name == "SPMM_ERR_INVALID_ARG"
    odd = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].reshape(q.shape)
    with pytest.raises(S.SpmmError) as e:
        S.spmm_execute_attn(P, odd, k, v, lists, o, lse)
    assert "aligned" in e.value.message
    with pytest.raises(S.SpmmError):
        S.spmm_execute(P, q[0, :, 0], o[0, :, 0])
    with pytest.raises(S.SpmmError):
        S.spmm_execute_sddmm(P, q[0, :, 0], o[0, :, 0], lse)


# ---- what stands where no query looks, far offsets, many items -------------

def test_keys_that_no_query_sees_may_hold_anything(S):
    """Keys below the length but past every query: NaN there changes nothing,
    and their gradients are zero."""
    for c in (case(nq=40, nk=256, hq=8, hk=2, d=128, q_block=64, blocks=4), case(nq=5, nk=256, hq=4, hk=4, q_block=1, blocks=4)):
        q, k, v, grad, g = inputs(c, 40)
        starts, lens = torch.tensor([70], dtype=torch.int32), torch.tensor([250], dtype=torch.int32)
        end = 70 + c["nq"]
        k[0, end:], v[0, end:] = float("nan"), float("inf")
        lists = torch.tensor([0, 1, 2, 3], dtype=torch.int32).expand(1, c["hk"], -(-c["nq"] // c["q_block"]), 4).contiguous()
        P = plan(S, c, backward=True)
        o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), lens.cuda(), starts.cuda(), P)
        dq, dk, dv = (torch.full_like(t, float("nan")).cuda() for t in (q, k, v))
        S.spmm_execute_attn_backward(P, grad.cuda(), q.cuda(), k.cuda(), v.cuda(), lists.cuda(), o, lse, dq, dk, dv,
                                     lens=lens.cuda(), starts=starts.cuda())
        want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, lists, lens, starts, None), grad.double())
        for name, got in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
            R.check(name, got, *want[name])
        assert (dk[:, end:] == 0).all() and (dv[:, end:] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nq,q_block", [(1, 1), (14, 1), (100, 16), (128, 64)])
def test_dq_of_few_keys_is_off_by_its_own_rounding(S, nq, q_block, dtype):
    """Up to two blocks: the rounding of dq, and errors of 32-bit sums; neither
    the rounding of o nor that of dS (kept to two steps) shows."""
    c = case(b=2, nq=nq, hq=4, hk=2, d=64, q_block=q_block, blocks=2, dtype=dtype)
    q, k, v, grad, g = inputs(c, 50 + nq)
    lists = torch.tensor([0, 1], dtype=torch.int32).expand(2, 2, -(-nq // q_block), 2).contiguous()
    P = plan(S, c, backward=True)
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), None, None, P)
    dq, dk, dv = (torch.full_like(t, float("nan")).cuda() for t in (q, k, v))
    S.spmm_execute_attn_backward(P, grad.cuda(), q.cuda(), k.cuda(), v.cuda(), lists.cuda(), o, lse, dq, dk, dv)
    q, k, v, grad = (t.double().permute(0, 2, 1, 3) for t in (q, k, v, grad))
    k, v = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    s = (q @ k.transpose(-1, -2) / 8).masked_fill(torch.ones(nq, nq).triu(1).bool(), -math.inf)
    p = torch.softmax(s, -1)
    dp = grad @ v.transpose(-1, -2)
    delta = (p * dp).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    want = ds @ k / 8
    u, e32 = torch.finfo(dtype).eps / 2, 2.0 ** -24
    tiny = torch.finfo(dtype).smallest_normal * u
    # relative errors of a weight: its score's 66 terms, exponents, the rounded lse
    ew = (2 * 66 * (q.abs() @ k.abs().transpose(-1, -2) / 8).amax(-1, keepdim=True) + 64) * e32
    edp = 66 * e32 * (grad.abs() @ v.abs().transpose(-1, -2))
    edelta = (p * (edp + (ew + 200 * e32) * dp.abs())).sum(-1, keepdim=True)
    eds = 1.02 * ((u * u + ew) * ds.abs() + p * (edp + edelta + 4 * e32 * (dp.abs() + delta.abs()))) + tiny * (p > 0)
    bound = (eds + 200 * e32 * ds.abs()) @ k.abs() / 8
    bound = (u + 4 * e32) * (want.abs() + bound) + bound + tiny
    R.check("dq", dq, want.permute(0, 2, 1, 3), bound.permute(0, 2, 1, 3))


def test_offsets_past_4_gib(S):
    """Pages, sequences and gradients that stand more than 2^32 bytes apart."""
    c = case(b=2, nq=70, nk=70, hq=4, hk=2, d=64, q_block=16, blocks=2)
    q, k, v, grad, g = inputs(c, 60)
    lists = random_lists(c, g).cuda()
    step = 2 ** 31 + 64  # elements
    room = torch.empty(step + 2 ** 20, dtype=c["dtype"], device="cuda")
    at = [0]

    def far(x):
        n = x[0].numel()
        y = room.as_strided(x.shape, (step, *x.stride()[1:]), at[0])
        at[0] += (n + 7) // 8 * 8
        y.copy_(x)
        return y

    outs = []
    for place in (lambda x: x, far):
        q1, k1, v1, g1 = (place(t.cuda()) for t in (q, k, v, grad))
        o, dq, dk, dv = (place(torch.zeros_like(t).cuda()) for t in (q, q, k, k))
        lse = torch.zeros((2, 4, 70), device="cuda")
        P = plan(S, c, backward=True)
        S.spmm_execute_attn(P, q1, k1, v1, lists, o, lse)
        S.spmm_execute_attn_backward(P, g1, q1, k1, v1, lists, o, lse, dq, dk, dv)
        values = torch.zeros((4, 2, 64), dtype=torch.int8, device="cuda")
        scale = torch.zeros((4, 2), device="cuda")
        S.spmm_execute_attn_pool(P, k1, values, scale)
        outs.append([t.contiguous() for t in (o, lse, dq, dk, dv, values, scale)])
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    assert outs[0][0][1].abs().sum() > 0
    # a cache whose second page stands past 2^32 bytes
    c = case(b=1, nq=3, nk=128, hq=4, hk=2, d=64, blocks=2)
    q, k, v, _, g = inputs(c, 61)
    table = torch.tensor([[1, 0]], dtype=torch.int32)
    pages = [x.reshape(2, PAGE, 2, 64).flip(0).contiguous().cuda() for x in (k, v)]
    starts = torch.tensor([125], dtype=torch.int32)
    at[0] = 0
    a = run_cache(S, c, q, *pages, table=table, starts=starts)
    b = run_cache(S, c, q, far(pages[0]), far(pages[1]), table=table, starts=starts)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, None, [128], [125], None))
    R.check("o", b[0], *want["o"])


def test_cache_strides(S):
    """Pages with their heads first, and K and V side by side in one page."""
    c = case(b=2, nq=4, nk=320, hq=8, hk=2, d=128, blocks=3)
    q, k, v, _, g = inputs(c, 62)
    kp, vp, table = paged(c, k, v, g)
    lens, starts = torch.tensor([320, 77], dtype=torch.int32), torch.tensor([316, 73], dtype=torch.int32)
    a = run_cache(S, c, q, kp, vp, table=table, lens=lens, starts=starts)
    both = torch.stack([kp, vp], 3).cuda()  # [pages, 64, heads, 2, dim]
    views = [(kp.cuda().transpose(1, 2).contiguous().transpose(1, 2), vp.cuda().transpose(1, 2).contiguous().transpose(1, 2)),
             (both[:, :, :, 0], both[:, :, :, 1])]
    for k1, v1 in views:
        assert not k1.is_contiguous()
        b = run_cache(S, c, q, k1, v1, table=table, lens=lens, starts=starts)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_backward_many_items(S):
    """More items than workgroups: the same bits as sequence by sequence."""
    c = case(b=8, nq=700, hq=16, hk=8, d=128, q_block=16, blocks=3)
    q, k, v, grad, g = inputs(c, 63)
    lists = random_lists(c, g, empty=0.1).cuda()
    lens = torch.tensor([700, 1, 650, 64, 65, 300, 700, 699], dtype=torch.int32).cuda()
    q, k, v, grad = (t.cuda() for t in (q, k, v, grad))

    def run(c, part):
        P = plan(S, c, backward=True)
        x = [t[part].contiguous() for t in (q, k, v, grad, lists, lens)]
        o, lse = run_forward(S, c, *x[:3], x[4], x[5], None, P)
        out = [torch.full_like(t, float("nan")) for t in x[:3]]
        for _ in range(2):  # the queues start anew
            S.spmm_execute_attn_backward(P, x[3], *x[:3], x[4], o, lse, *out, lens=x[5])
        return out

    whole = run(c, slice(0, 8))
    for i in range(8):
        for x, y in zip(whole, run(dict(c, b=1), slice(i, i + 1))):
            assert torch.equal(x[i:i + 1], y), i


def test_plan_out_of_memory(S, monkeypatch):
    """Every allocation of a plan that fails: OUT_OF_MEMORY, and the next plan works."""
    n = 1
    while True:
        monkeypatch.setenv("SPMM_TEST_FAIL_ALLOC", str(n))
        try:
            plan(S, case(b=1, nq=2, nk=4096, hq=4, hk=2, q_block=1, blocks=64), backward=True)
            break
        except S.SpmmError as e:
            assert e.name == "SPMM_ERR_OUT_OF_MEMORY"
        n += 1
    assert n > 6
    monkeypatch.delenv("SPMM_TEST_FAIL_ALLOC")
    plan(S, case(), backward=True)


# ---- lists that share a row tile -------------------------------------------

PACKED = [
    case(b=2, nq=1100, hq=32, hk=2, d=128, q_block=1, blocks=5),
    case(b=1, nq=1050, hq=12, hk=4, d=64, q_block=1, blocks=3, dtype=torch.float16),
    case(b=1, nq=2100, hq=8, hk=4, d=64, q_block=1, blocks=4),
    case(b=1, nq=2060, nk=500, hq=4, hk=4, d=128, q_block=2, blocks=7, dtype=torch.float16),
]


def packed_lists(c, g):
    """Lists of neighbours that share blocks, with gaps, some empty, some
    naming a block twice, some past the end."""
    lists = random_lists(c, g, empty=0.1)
    lists[:, :, 1::3] = lists[:, :, :-1:3][:, :, :lists[:, :, 1::3].shape[2]]
    lists[:, :, ::5, 1] = lists[:, :, ::5, 0]
    lists[:, :, ::7, -1] = 2 ** 31 - 1
    lists[:, :, ::11, 0] = -1
    return lists


@pytest.mark.parametrize("n", range(len(PACKED)))
def test_lists_that_share_a_tile(S, n):
    c = PACKED[n]
    assert c["b"] * c["hk"] * -(-c["nq"] // c["q_block"]) >= 4096
    q, k, v, grad, g = inputs(c, 900 + n)
    lists = packed_lists(c, g)
    nk = c["nk"]
    lens = torch.tensor([nk, nk - 77][:c["b"]], dtype=torch.int32)
    starts = torch.tensor([nk - c["nq"], -5][:c["b"]], dtype=torch.int32).clamp(max=20)
    P = plan(S, c, backward=True)
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), lens.cuda(), starts.cuda(), P)
    dq, dk, dv = (torch.full_like(t, float("nan")).cuda() for t in (q, k, v))
    S.spmm_execute_attn_backward(P, grad.cuda(), q.cuda(), k.cuda(), v.cuda(), lists.cuda(), o, lse, dq, dk, dv,
                                 lens=lens.cuda(), starts=starts.cuda())
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, lists, lens, starts, None), grad.double())
    for name, got in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        R.check(name, got, *want[name])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_neighbours_list_does_not_spoil_a_row(S, bad):
    """A block with values that are no numbers, named by one list of a tile:
    the other lists' rows come out as without it."""
    c = case(b=2, nq=1100, hq=32, hk=2, d=128, q_block=1, blocks=2)
    q, k, v, grad, g = inputs(c, 950)
    starts = torch.tensor([0, 0], dtype=torch.int32)
    lists = torch.zeros((2, 2, 1100, 2), dtype=torch.int32)
    lists[..., 1] = -1
    lists[:, :, 901::9, 1] = 3
    clean = [t.clone() for t in (k, v)]
    k[:, 200], v[:, 210] = bad, bad  # in block 3
    sees3 = (lists[..., 1] == 3).repeat_interleave(16, 1)  # [b, hq, nq]
    outs = []
    for k1, v1 in ((k, v), clean):
        P = plan(S, c, backward=True)
        o, lse = run_forward(S, c, q.cuda(), k1.cuda(), v1.cuda(), lists.cuda(), None, starts.cuda(), P)
        dq, dk, dv = (torch.full_like(t, float("nan")).cuda() for t in (q, k, v))
        S.spmm_execute_attn_backward(P, grad.cuda(), q.cuda(), k1.cuda(), v1.cuda(), lists.cuda(), o, lse, dq, dk, dv)
        outs.append([o.cpu().transpose(1, 2), lse.cpu(), dq.cpu().transpose(1, 2)])
    for x, y in zip(*outs):
        assert torch.isfinite(y).all()
        assert torch.equal(x[~sees3], y[~sees3])
    assert not torch.isfinite(outs[0][0][sees3]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nq,q_block,hk", [(1, 1, 4), (2, 64, 1), (6, 16, 2), (100, 4, 4), (128, 64, 2)])
def test_dk_dv_of_short_sequences_are_off_by_their_own_rounding(S, nq, q_block, hk, dtype):
    """Up to 128 queries: the rounding of dk and dv, and errors of 32-bit sums."""
    c = case(b=2, nq=nq, hq=4, hk=hk, d=128, q_block=q_block, blocks=2, dtype=dtype)
    q, k, v, grad, g = inputs(c, 970 + nq)
    lists = torch.tensor([0, 1], dtype=torch.int32).expand(2, hk, -(-nq // q_block), 2).contiguous()
    P = plan(S, c, backward=True)
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), None, None, P)
    dq, dk, dv = (torch.full_like(t, float("nan")).cuda() for t in (q, k, v))
    S.spmm_execute_attn_backward(P, grad.cuda(), q.cuda(), k.cuda(), v.cuda(), lists.cuda(), o, lse, dq, dk, dv)
    q, k, v, grad = (t.double().permute(0, 2, 1, 3) for t in (q, k, v, grad))
    k, v = k.repeat_interleave(4 // hk, 1), v.repeat_interleave(4 // hk, 1)
    scale = 1.0 / math.sqrt(128)
    s = (scale * (q @ k.transpose(-1, -2))).masked_fill(torch.ones(nq, nq).triu(1).bool(), -math.inf)
    p = torch.softmax(s, -1)
    dp = grad @ v.transpose(-1, -2)
    delta = (p * dp).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    u, e32 = torch.finfo(dtype).eps / 2, 2.0 ** -24
    tiny = torch.finfo(dtype).smallest_normal * u
    # as for dq: a weight's score of 130 terms, exponents, the rounded lse
    ew = (2 * 130 * scale * (q.abs() @ k.abs().transpose(-1, -2)).amax(-1, keepdim=True) + 64) * e32
    edp = 130 * e32 * (grad.abs() @ v.abs().transpose(-1, -2))
    edelta = (p * (edp + (ew + 400 * e32) * dp.abs())).sum(-1, keepdim=True)
    on = (p > 0).double()
    eds = 1.02 * ((u * u + ew) * ds.abs() + p * (edp + edelta + 4 * e32 * (dp.abs() + delta.abs()))) + tiny * on
    ep = 1.02 * (u * u + ew) * p + tiny * on
    rows = 4 // hk * nq

    def per_key(x):
        return x.reshape(2, hk, 4 // hk, nq, 128).sum(2).permute(0, 2, 1, 3)

    for name, got, w, e, x, f in (("dk", dk, ds, eds, q, scale), ("dv", dv, p, ep, grad, 1.0)):
        want = per_key(f * (w.transpose(-1, -2) @ x))
        off = per_key(f * ((e + rows * e32 * w.abs()).transpose(-1, -2) @ x.abs()))
        R.check(name, got, want, (u + 4 * e32) * (want.abs() + off) + off + tiny)


MANY = [  # more tiles of 128 rows than CUs: a workgroup has no second group of waves for them
    case(nq=521, hq=40, hk=8, q_block=16, blocks=5), case(b=4, nq=300, hq=28, hk=14, d=128, dtype=torch.float16),
    case(b=4, nq=570, nk=600, hq=16, hk=2, blocks=3, dtype=torch.float16), case(b=2, nq=545, hq=24, hk=8, d=128, q_block=32),
]


@pytest.mark.parametrize("kind", ["full", "ragged", "odd"])
@pytest.mark.parametrize("n", range(len(MANY)))
def test_many_tiles_of_many_rows(S, n, kind):
    c = MANY[n]
    rows = c["q_block"] * (c["hq"] // c["hk"])
    assert rows > 64 and c["b"] * c["hk"] * -(-c["nq"] // c["q_block"]) * -(-rows // 128) > 256
    q, k, v, grad, g = inputs(c, 1100 + n)
    lens, starts = lengths(c, g, kind)
    lists = random_lists(c, g, empty=0.2)
    P = plan(S, c, backward=True)
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), lens.cuda(), starts.cuda(), P)
    dq, dk, dv = (torch.full_like(t, float("nan")).cuda() for t in (q, k, v))
    S.spmm_execute_attn_backward(P, grad.cuda(), q.cuda(), k.cuda(), v.cuda(), lists.cuda(), o, lse, dq, dk, dv,
                                 lens=lens.cuda(), starts=starts.cuda())
    w = R.sees(c, lists, lens, starts, None)
    want = R.attention(c, q.double(), k.double(), v.double(), w, grad.double())
    for name, got in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        R.check(name, got, *want[name])


# ---- queries that see nothing of a block -----------------------------------

QUIET = [
    case(nq=64, nk=192, hq=4, hk=2, d=128, q_block=64, blocks=1), case(nq=48, nk=128, hq=3, hk=3, q_block=16, blocks=2),
    case(nq=150, nk=256, hq=8, hk=1, d=64, q_block=4, blocks=1, dtype=torch.float16),
]


@pytest.mark.parametrize("n", range(len(QUIET)))
def test_queries_without_keys_take_no_part(S, n):
    """Lists that name the second block only: the queries before it see no key,
    and what stands in their q and grad reaches no gradient."""
    c = QUIET[n]
    q, k, v, grad, g = inputs(c, 1200 + n)
    starts, lens = torch.tensor([37], dtype=torch.int32), torch.tensor([c["nk"] - 3], dtype=torch.int32)
    lists = torch.full((1, c["hk"], -(-c["nq"] // c["q_block"]), c["blocks"]), -1, dtype=torch.int32)
    lists[..., 0] = 1
    quiet = PAGE - 37
    q[0, :quiet:2], q[0, 1:quiet:2] = float("nan"), float("inf")
    grad[0, :quiet:2], grad[0, 1:quiet:2] = float("inf"), float("nan")
    P = plan(S, c, backward=True)
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), lens.cuda(), starts.cuda(), P)
    dq, dk, dv = (torch.full_like(t, float("nan")).cuda() for t in (q, k, v))
    S.spmm_execute_attn_backward(P, grad.cuda(), q.cuda(), k.cuda(), v.cuda(), lists.cuda(), o, lse, dq, dk, dv,
                                 lens=lens.cuda(), starts=starts.cuda())
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, lists, lens, starts, None), grad.double())
    for name, got in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        R.check(name, got, *want[name])
    assert (o[:, :quiet] == 0).all() and (dq[:, :quiet] == 0).all() and (dk[:, PAGE:] != 0).any()


def test_queries_before_a_block_do_not_reach_it(S):
    """Queries that see the first block alone, in one list with later ones: no
    number of theirs reaches the gradients of the second block."""
    c = case(nq=64, nk=128, hq=4, hk=2, d=128, q_block=64, blocks=2)
    q, k, v, grad, g = inputs(c, 1210)
    starts = torch.tensor([40], dtype=torch.int32, device="cuda")
    lists = torch.tensor([0, 1], dtype=torch.int32).expand(1, 2, 1, 2).contiguous().cuda()
    outs = []
    for bad in (False, True):
        if bad:
            q[0, 3], grad[0, 20] = float("nan"), float("inf")
        P = plan(S, c, backward=True)
        x = [t.cuda() for t in (q, k, v, grad)]
        o, lse = run_forward(S, c, *x[:3], lists, None, starts, P)
        dq, dk, dv = (torch.full_like(t, float("nan")) for t in x[:3])
        S.spmm_execute_attn_backward(P, x[3], *x[:3], lists, o, lse, dq, dk, dv, starts=starts)
        outs.append((dk[:, PAGE:], dv[:, PAGE:]))
    for x, y in zip(*outs):
        assert torch.isfinite(x).all() and torch.equal(x, y)


# ---- gradients of f16 whose dS pass its range ------------------------------

WIDE = [  # a list of many rows, short and longer sequences; of few rows, four waves, a wave, several lists to a tile
    case(nq=64, d=128, blocks=1), case(nq=200, hk=1, blocks=4), case(nq=300, hq=8, hk=8, q_block=1, blocks=5),
    case(nq=2100, hq=2, hk=2, q_block=1, blocks=33), case(nq=1100, hq=8, hk=4, q_block=1, blocks=18, d=128),
]


@pytest.mark.parametrize("step", [1.0, 2.0 ** -18])
@pytest.mark.parametrize("n", range(len(WIDE)))
def test_gradients_of_f16_with_dS_past_its_range(S, n, step):
    """Values that are large and keys and queries that are not: dS goes to many
    times 65504 where every gradient fits; the same with gradients 2^18 smaller."""
    c = dict(WIDE[n], dtype=torch.float16)
    q, k, v, grad, g = inputs(c, 1300 + n)
    q, k, v, grad = (q.float() / 8).half(), (k.float() / 8).half(), v * 64, (grad.float() * 1000 * step).half()
    nqb, nkb = -(-c["nq"] // c["q_block"]), -(-c["nk"] // PAGE)
    lists = torch.arange(nkb, dtype=torch.int32).expand(1, c["hk"], nqb, nkb).contiguous()
    P = plan(S, c, backward=True)
    o, lse = run_forward(S, c, q.cuda(), k.cuda(), v.cuda(), lists.cuda(), None, None, P)
    dq, dk, dv = (torch.full_like(t, float("nan")).cuda() for t in (q, k, v))
    S.spmm_execute_attn_backward(P, grad.cuda(), q.cuda(), k.cuda(), v.cuda(), lists.cuda(), o, lse, dq, dk, dv)
    w = torch.ones(c["nq"], c["nk"]).tril().double().expand(1, c["hk"], -1, -1)
    want = R.attention(c, q.double(), k.double(), v.double(), w, grad.double())
    for x in ("dq", "dk", "dv"):
        assert want[x][0].abs().max() < 65504
    if step == 1.0:  # the second query's dS for its two keys, in one head: of opposite signs, p (1 - p) grad . (v0 - v1)
        gt, vt = grad[0, 1].double(), v[0, :2].repeat_interleave(c["hq"] // c["hk"], 1).double()
        assert ((gt * (vt[0] - vt[1])).sum(-1).abs().max() / 4) > 2 * 65504
    for name, got in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        R.check(name, got, *want[name])


# ---- keys that few rows read, in long sequences ----------------------------

def own_rounding(c, q, k, v, grad, w):
    """dq, dk and dv with bounds that hold their own rounding and the errors of
    32-bit sums alone: P, dS and delta are kept to two steps of their rounding."""
    u, e32 = torch.finfo(c["dtype"]).eps / 2, 2.0 ** -24
    tiny = torch.finfo(c["dtype"]).smallest_normal * u
    d, n, group, scale = c["d"], c["nk"], c["hq"] // c["hk"], 1.0 / math.sqrt(c["d"])
    q, k, v, grad = (t.double().permute(0, 2, 1, 3) for t in (q, k, v, grad))
    k, v, w = (t.repeat_interleave(group, 1) for t in (k, v, w))
    on = w > 0
    k, v = (torch.where(on.any(-2)[..., None], t, 0.0) for t in (k, v))
    q, grad = (torch.where(on.any(-1)[..., None], t, 0.0) for t in (q, grad))
    s = (scale * (q @ k.transpose(-1, -2))).masked_fill(~on, -math.inf)
    p = torch.where(on, torch.softmax(s, -1), 0.0)
    dp = grad @ v.transpose(-1, -2)
    delta = (p * dp).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    # relative errors of a weight: its score's d + 2 terms, exponents, the rounded lse
    ew = torch.where(on, 2 * (d + 2) * scale * (q.abs() @ k.abs().transpose(-1, -2)), 0.0).amax(-1, keepdim=True)
    ew = (ew + 64 + 8 * torch.where(on, s, 0.0).abs().amax(-1, keepdim=True)) * e32
    edp = (d + 2) * e32 * (grad.abs() @ v.abs().transpose(-1, -2))
    edelta = (p * (edp + (ew + 2 * n * e32) * dp.abs())).sum(-1, keepdim=True)
    eds = 1.02 * ((u * u + ew) * ds.abs() + p * (edp + edelta + 4 * e32 * (dp.abs() + delta.abs()))) + tiny * on
    ep = 1.02 * (u * u + ew) * p + tiny * on

    def per_key(x):
        return x.reshape(c["b"], c["hk"], group, *x.shape[2:]).sum(2)

    rows, out = group * c["nq"], {}
    for name, want, off in (
            ("dq", scale * (ds @ k), scale * ((eds + n * e32 * ds.abs()) @ k.abs())),
            ("dk", per_key(scale * (ds.transpose(-1, -2) @ q)), per_key(scale * ((eds + rows * e32 * ds.abs()).transpose(-1, -2) @ q.abs()))),
            ("dv", per_key(p.transpose(-1, -2) @ grad), per_key((ep + rows * e32 * p).transpose(-1, -2) @ grad.abs()))):
        out[name] = (want.permute(0, 2, 1, 3), ((u + 4 * e32) * (want.abs() + off) + off + tiny).permute(0, 2, 1, 3))
    return out


def gradients(S, c, q, k, v, grad, lists, lens=None):
    P = plan(S, c, backward=True)
    x = [t.cuda() for t in (q, k, v, grad, lists)]
    lens = dev(lens)
    o, lse = run_forward(S, c, *x[:3], x[4], lens, None, P)
    out = [torch.full_like(t, float("nan")) for t in x[:3]]
    S.spmm_execute_attn_backward(P, x[3], *x[:3], x[4], o, lse, *out, lens=lens)
    return dict(zip(("dq", "dk", "dv"), out), o=o, lse=lse)


@pytest.mark.parametrize("hk,q_block,dtype", [(2, 64, torch.bfloat16), (1, 16, torch.bfloat16), (2, 1, torch.float16)])
def test_short_sequences_next_to_a_long_one(S, hk, q_block, dtype):
    """Sequences of 10 to 128 tokens in tensors of 500: dq, dk and dv are off by
    their own rounding, as they are alone."""
    c = case(b=6, nq=500, hq=2, hk=hk, d=128, q_block=q_block, blocks=2, dtype=dtype)
    q, k, v, grad, g = inputs(c, 1400 + q_block)
    lens = torch.tensor([10, 33, 64, 100, 115, 128], dtype=torch.int32)
    lists = torch.tensor([0, 1], dtype=torch.int32).expand(6, hk, -(-500 // q_block), 2).contiguous()
    got = gradients(S, c, q, k, v, grad, lists, lens)
    want = own_rounding(c, q, k, v, grad, R.sees(c, lists, lens, [0] * 6, None))
    for name in ("dq", "dk", "dv"):
        R.check(name, got[name], *want[name])


@pytest.mark.parametrize("nq,q_block,hq,hk,dtype", [(700, 64, 8, 8, torch.bfloat16), (700, 16, 4, 1, torch.float16), (1300, 64, 4, 1, torch.bfloat16)])
def test_blocks_that_few_rows_read(S, nq, q_block, hq, hk, dtype):
    """A long sequence whose lists name their own block: up to 256 rows read it."""
    c = case(nq=nq, hq=hq, hk=hk, d=128, q_block=q_block, blocks=1, dtype=dtype)
    q, k, v, grad, g = inputs(c, 1410 + q_block)
    nqb = -(-nq // q_block)
    lists = (torch.arange(nqb, dtype=torch.int32) * q_block // PAGE).reshape(1, 1, nqb, 1).expand(1, hk, nqb, 1).contiguous()
    got = gradients(S, c, q, k, v, grad, lists)
    want = own_rounding(c, q, k, v, grad, R.sees(c, lists, [nq], [0], None))
    for name in ("dq", "dk", "dv"):
        R.check(name, got[name], *want[name])


@pytest.mark.parametrize("hq,d,dtype", [(8, 64, torch.bfloat16), (16, 128, torch.float16)])
def test_a_short_list_keeps_its_delta_next_to_long_ones(S, hq, d, dtype):
    """Lists of one and two blocks that share a tile with lists of seven: their
    dq is off by its own rounding."""
    c = case(nq=1100, hq=hq, hk=8, d=d, q_block=1, blocks=8, dtype=dtype)
    q, k, v, grad, g = inputs(c, 1430)
    nkb, t = -(-c["nq"] // PAGE), torch.arange(c["nq"])
    lists = torch.full((1, 8, c["nq"], 8), -1, dtype=torch.int32)
    for j in range(7):
        lists[..., j] = (t[None] * (j + 1) + 5 * torch.arange(8)[:, None]) % nkb
    lists = lists.sort(-1).values
    lists[:, :, ::2, :6] = -1  # a block, and the query's own
    lists[:, :, ::2, 7] = (t[::2] // PAGE).int()
    lists[:, :, ::4, 6] = nkb - 1 - lists[:, :, ::4, 6] % 4  # most see nothing of it
    got = gradients(S, c, q, k, v, grad, lists)
    w = R.sees(c, lists, [c["nq"]], [0], None)
    want = own_rounding(c, q, k, v, grad, w.clamp(max=1.0))["dq"]
    once = (w[0].amax(-1) <= 1).repeat_interleave(hq // 8, 0).T  # no block named twice
    short = once & (t % 2 == 0)[:, None]
    assert short.sum() > 300 * hq // 2
    R.check("dq", got["dq"].cpu()[0][short], want[0][0][short], want[1][0][short])


@pytest.mark.parametrize("nq,hq,listed", [(4, 4, False), (40, 8, True), (64, 16, False)])
def test_tree_keys_past_every_bit_may_hold_anything(S, nq, hq, listed):
    """A mask has 64 bits: keys 64 and more past the text are seen by no drafted token."""
    c = case(b=2, nq=nq, nk=640, hq=hq, hk=2, d=128, blocks=10)
    q, k, v, _, g = inputs(c, 1440 + nq)
    starts, lens = torch.tensor([130, 400], dtype=torch.int32), torch.tensor([400, 640], dtype=torch.int32)
    tree = torch.randint(-2 ** 63, 2 ** 63 - 1, (2, nq), generator=g)
    for i in range(2):
        at = int(starts[i]) + 64
        k[i, at::2], k[i, at + 1::2] = float("nan"), float("inf")
        v[i, at::2], v[i, at + 1::2] = float("inf"), float("nan")
    kp, vp, table = paged(c, k, v, g)
    lists = torch.arange(10, dtype=torch.int32).expand(2, 2, 1, 10).contiguous() if listed else None
    o, lse = run_cache(S, c, q, kp, vp, table=table, lists=lists, lens=lens, starts=starts, tree=tree)
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, lists, lens, starts, tree))
    R.check("o", o, *want["o"])
    R.check("lse", lse, *want["lse"])


# ---- lists and sequences that are cut into ranges --------------------------

def ranges(P, c, listed):
    """Ranges of a list, or of a whole sequence (then the larger of the two)."""
    if listed:
        rows = min(c["q_block"], c["nq"]) * (c["hq"] // c["hk"])
        tiles = -(-rows // P.info()["tile_m"])
        return P.info()["grid"] // (c["b"] * c["hk"] * tiles)
    return P.info()["workspace_bytes"] // (c["b"] * c["hq"] * c["nq"] * (c["d"] * 4 + 8))


TREES = [  # row tiles of 32, 64, 128, 256 rows, several of 128 and of 256
    case(b=3, nq=4, nk=6000, hq=8, hk=2, d=128, blocks=2), case(b=2, nq=12, nk=5000, hq=4, hk=1, blocks=2),
    case(b=3, nq=24, nk=4500, hq=8, hk=2, d=128, blocks=2), case(b=2, nq=24, nk=5000, hq=8, hk=1, blocks=2, dtype=torch.float16),
    case(b=1, nq=24, nk=7000, hq=16, hk=1, d=128, blocks=2), case(b=2, nq=64, nk=4200, hq=16, hk=1, d=128, blocks=2),
]


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("n", range(len(TREES)))
def test_cache_tree_in_ranges(S, n, listed):
    c = dict(TREES[n], blocks=48) if listed else TREES[n]
    assert ranges(plan(S, c), c, listed) > 1, "the case must be cut"
    q, k, v, _, g = inputs(c, 1500 + n)
    lens = torch.tensor([c["nk"], c["nk"] // 3 + 5, c["nq"] - 1][:c["b"]], dtype=torch.int32)
    starts = lens - c["nq"]
    tree = torch.randint(-2 ** 63, 2 ** 63 - 1, (c["b"], c["nq"]), generator=g)
    kp, vp, table = paged(c, k, v, g)
    lists = random_lists(c, g) if listed else None
    if listed:  # with the drafted tokens' own block, and a gap before it
        lists[..., -2], lists[..., -1] = -1, ((lens - 1) // PAGE)[:, None, None]
    o, lse = run_cache(S, c, q, kp, vp, table=table, lists=lists, lens=lens, starts=starts, tree=tree)
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, lists, lens, starts, tree))
    R.check("o", o, *want["o"])
    R.check("lse", lse, *want["lse"])


LISTED = [  # a row, few rows, 32 rows to a list; long lists
    case(b=4, nq=1, nk=8192, hq=2, hk=2, d=128, blocks=32), case(b=4, nq=1, nk=8000, hq=8, hk=2, d=128, blocks=32, dtype=torch.float16),
    case(b=2, nq=5, nk=8192, hq=4, hk=2, blocks=48), case(b=1, nq=2, nk=3000, hq=16, hk=1, d=128, blocks=47),
    case(b=2, nq=1, nk=30000, hq=4, hk=1, blocks=300),
]


@pytest.mark.parametrize("kind", ["full", "ragged", "odd"])
@pytest.mark.parametrize("n", range(len(LISTED)))
def test_lists_of_few_rows_in_ranges(S, n, kind):
    """Lists that end inside a range, with gaps, doubles and blocks past the
    end, empty ones, and pages that are none."""
    c = LISTED[n]
    assert ranges(plan(S, c), c, True) > 1, "the case must be cut"
    q, k, v, _, g = inputs(c, 1520 + n)
    lens, starts = lengths(c, g, kind)
    lists = random_lists(c, g, empty=0.2)
    lists[:, 0, :, 3], lists[:, 0, :, 9] = -1, 2 ** 31 - 1
    lists[:, -1, :, 1] = lists[:, -1, :, 0]
    kp, vp, table = paged(c, k, v, g)
    ok = torch.ones(table.shape)
    table[0, 2], table[-1, 5], ok[0, 2], ok[-1, 5] = -1, kp.shape[0], 0, 0
    o, lse = run_cache(S, c, q, kp, vp, table=table, lists=lists, lens=lens, starts=starts)
    want = R.attention(c, q.double(), k.double(), v.double(), R.sees(c, lists, lens, starts, None, ok))
    R.check("o", o, *want["o"])
    R.check("lse", lse, *want["lse"])
