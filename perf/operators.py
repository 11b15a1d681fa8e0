"""Cases for timing block-sparse attention: the choice of key blocks by a
cheap score, attention over the chosen blocks (forward, and forward with the
gradients), and attention of new or drafted tokens over a cache.

Sequences are cut into blocks (pages) of 64 keys.  A list names the blocks
that a query block of q_block tokens reads for one key/value head, ascending,
padded with -1.  Query t of a sequence stands at position start + t; a key is
seen when its position is below the sequence's length, at most the query's
own, and in a block of the list.  A cache holds pages of 64 keys reached
through a table; drafted tokens stand in its last positions and see one
another by the bits of a tree mask.
"""
import math

import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---- cases -----------------------------------------------------------------

def _case(name, op, **kw):
    c = {"op": op, "batch": 1, "len": 0, "tokens": 0, "heads_q": 32, "heads_kv": 8, "dim": 128,
         "q_block": 64, "blocks": 16, "dtype": "bf16", "ragged": False, "tree": False, "sparse": False}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # serving: one decode step of 32 ragged sequences picks 32 pages of up to 256
        _case("select step 32x16k", "select", batch=32, len=16384, tokens=1, blocks=32, ragged=True),
        # prefill: a 32k prompt, one list for 64 queries
        _case("select prompt 32k", "select", len=32768, blocks=32),
        # short ragged prompts with small heads and three query heads to a key head
        _case("forward ragged 3x777", "forward", batch=3, len=777, heads_q=6, heads_kv=2, dim=64, q_block=16,
              blocks=4, dtype="f16", ragged=True),
        # prefill of a 32k prompt reading 2048 keys a query
        _case("forward prompt 32k", "forward", len=32768, blocks=32),
        # every query has its own list, 16 query heads share a key head
        _case("forward per query 8k", "forward", len=8192, heads_q=64, heads_kv=4, q_block=1),
        # training on short ragged texts, as many key heads as query heads
        _case("train ragged 2x1000", "train", batch=2, len=1000, heads_q=4, heads_kv=4, dim=64, q_block=32,
              blocks=4, ragged=True),
        # training on a long text, 64 queries to a list
        _case("train 16k", "train", len=16384),
        # training with a list for each query
        _case("train per query 4k", "train", len=4096, heads_q=32, heads_kv=2, q_block=1),
        # one user's next token: latency counts
        _case("cache step 1x4097", "cache", batch=1, len=4097, tokens=1),
        # a full batch of long ragged sequences, every page read
        _case("cache step 32x32k", "cache", batch=32, len=32768, tokens=1, ragged=True),
        # the same kind of batch reading 32 chosen pages a key head
        _case("cache chosen 64x16k", "cache", batch=64, len=16384, tokens=1, blocks=32, ragged=True, sparse=True),
        # 24 drafted tokens of a tree, checked at once
        _case("cache tree 16x8k", "cache", batch=16, len=8192, tokens=24, ragged=True, tree=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "forward", "train", "cache"])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    group = min(group, 64 // kv)
    dtype = "bf16" if op == "train" else rng.choice(["bf16", "bf16", "f16"])
    ragged = rng.random() < 0.5
    if op == "cache" or (op == "select" and rng.random() < 0.5):
        tokens = rng.choice([1, 1, 1, rng.randint(2, 12), rng.randint(13, 64)])
        batch = _log(rng, 1, 48)
        length = max(tokens, _log(rng, 1, min(32768, 700000 // batch)))
        return _case(None, op, batch=batch, len=length, tokens=tokens, heads_q=kv * group, heads_kv=kv, dim=dim,
                     blocks=rng.randint(2, 48), dtype=dtype, ragged=ragged, tree=op == "cache" and tokens > 1,
                     sparse=op == "cache" and rng.random() < 0.4)
    q_block = rng.choice([1, 4, 16, 32, 64])
    batch = _log(rng, 1, 4)
    most = (16384 if q_block >= 16 else 4096) // batch
    return _case(None, op, batch=batch, len=_log(rng, 1, most), heads_q=kv * group, heads_kv=kv, dim=dim,
                 q_block=q_block, blocks=rng.randint(2, 20), dtype=dtype, ragged=ragged)


def _lens(c):
    """Lengths of the sequences: they differ where the case is ragged."""
    least = max(1, c["tokens"])
    return [max(least, c["len"] - (i * 2654435761 % 997) * c["len"] // 1300 if c["ragged"] else c["len"])
            for i in range(c["batch"])]


def _geometry(c):
    """(queries a sequence, tokens of a list, query blocks, key blocks)"""
    if c["tokens"]:
        return c["tokens"], 64, 1, -(-c["len"] // PAGE)
    return c["len"], c["q_block"], -(-c["len"] // c["q_block"]), -(-c["len"] // PAGE)


def work(case):
    c, d = case, case["dim"]
    hq, hk, lens = c["heads_q"], c["heads_kv"], _lens(case)
    elem = 2
    pairs = keys = scored = blocks = 0  # (query, key) pairs of a query head; keys read, scored and kept of a key head
    for n in lens:
        nb = -(-n // PAGE)
        if c["tokens"]:
            t = c["tokens"]
            read = min(n, c["blocks"] * PAGE) if (c["sparse"] or c["op"] == "select") else n
            pairs += t * (read - t) + t * (t + 1) // 2
            keys += read
            scored += nb
            blocks += 1
        else:
            for j in range(nb):  # queries 64 j .. all read min(j + 1, blocks) blocks, the last one up to themselves
                rows = min(PAGE, n - j * PAGE)
                pairs += rows * (min(j + 1, c["blocks"]) - 1) * PAGE + rows * (rows + 1) // 2
                scored += -(-rows // c["q_block"]) * (j + 1)
            keys += n
            blocks += nb
    queries = sum(c["tokens"] or n for n in lens)
    if c["op"] == "select":
        lists = (c["batch"] if c["tokens"] else sum(-(-n // c["q_block"]) for n in lens)) * hk * c["blocks"] * 4
        tables = (scored if c["tokens"] else blocks) * hk * (d + 4)
        fresh = (c["batch"] * PAGE if c["tokens"] else keys) * hk * d * elem
        return {"bytes": float(queries * hq * d * elem + fresh + tables + lists),
                "flops": float(2 * d * hk * scored + (queries * hq + fresh // (d * elem)) * d)}
    once = queries * hq * d * elem + 2 * keys * hk * d * elem
    if c["op"] == "train":
        return {"bytes": float(3 * queries * hq * d * elem + queries * hq * 4 + queries * hq * d * elem
                               + 4 * keys * hk * d * elem), "flops": float(14 * d * hq * pairs)}
    return {"bytes": float(once + queries * hq * (d * elem + 4)), "flops": float(4 * d * hq * pairs)}


# ---- inputs ----------------------------------------------------------------

def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype, d, hq, hk, b = DTYPES[c["dtype"]], c["dim"], c["heads_q"], c["heads_kv"], c["batch"]
    nq, q_block, nqb, nkb = _geometry(c)
    lens = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
    starts = (lens - nq) if c["tokens"] else torch.zeros_like(lens)
    s = {"case": c, "lens": lens, "starts": starts.contiguous(), "scale": 1.0 / math.sqrt(d)}
    # texts drift from topic to topic: keys and queries of a stretch of 128
    # tokens share a part, and topics come back
    stretch = 128
    topics = 0.5 * torch.randn((64, hk, d), generator=g, device="cuda")
    length = nkb * PAGE if c["tokens"] else c["len"]
    which = torch.randint(0, 64, (b, -(-length // stretch)), generator=g, device="cuda")
    at = torch.arange(length, device="cuda") // stretch
    k = (torch.randn((b, length, hk, d), generator=g, device="cuda") + topics[which[:, at]]).to(dtype)
    v = _normal(g, (b, length, hk, d), dtype)
    pos = (starts[:, None].long() + torch.arange(nq, device="cuda")).clamp(0, length - 1)
    part = topics[which.gather(1, pos // stretch)].repeat_interleave(hq // hk, dim=2)
    s["q"] = (torch.randn((b, nq, hq, d), generator=g, device="cuda") + part).to(dtype)
    del part
    if c["tokens"]:  # pages in an order of their own
        order = torch.randperm(b * nkb, generator=g, device="cuda")
        s["table"] = order.reshape(b, nkb).to(torch.int32)
        s["k"], s["v"] = torch.empty((2, b * nkb, PAGE, hk, d), dtype=dtype, device="cuda")
        s["k"][order] = k.reshape(b * nkb, PAGE, hk, d)
        s["v"][order] = v.reshape(b * nkb, PAGE, hk, d)
    else:
        s["k"], s["v"], s["table"] = k, v, None
    del k, v
    if c["op"] == "train":
        s["grad"] = _normal(g, s["q"].shape, dtype)
    if c["tree"]:  # each drafted token hangs below an earlier one, or below the text
        parent = (torch.rand((b, nq), generator=g, device="cuda") * torch.arange(nq, device="cuda")).long()
        bits = torch.zeros((b, nq), dtype=torch.int64, device="cuda")
        bits[:, 0] = 1
        for t in range(1, nq):
            bits[:, t] = bits.gather(1, parent[:, t:t + 1])[:, 0] | (1 << t if t < 63 else -(1 << 63))
        s["tree"] = bits
    else:
        s["tree"] = None
    # what a cheap score has chosen before, or keeps of the pages
    s["pooled"] = torch.zeros((b * nkb, hk, d), dtype=torch.int8, device="cuda")
    s["pooled_scale"] = torch.zeros((b * nkb, hk), dtype=torch.float32, device="cuda")
    s["lists"] = torch.full((b, hk, nqb, c["blocks"]), -1, dtype=torch.int32, device="cuda")
    s["first"] = None
    if c["op"] != "cache" or c["sparse"]:
        _pool(s)
    if c["op"] == "select":
        if c["tokens"]:
            s["first"] = s["starts"]  # the pages before the new tokens are pooled already
    elif c["op"] != "cache" or c["sparse"]:
        _select(s)
    if own:
        import sparse_dense_matrix_amd as S
        s["plan"] = S.spmm_plan_attn(
            b, nq, nkb * PAGE if c["tokens"] else c["len"], hq, hk, d, dtype={"bf16": S.BF16, "f16": S.F16}[c["dtype"]],
            q_block=q_block, max_blocks=c["blocks"], sink_blocks=1, local_blocks=1, backward=c["op"] == "train")
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((b, hq, nq), dtype=torch.float32, device="cuda")
        if c["op"] == "train":
            s["dq"], s["dk"], s["dv"] = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    return s


# ---- plain forms -----------------------------------------------------------

def _pool(s):
    """Mean keys of the blocks in 8 bits with a scale, written where the block's page stands.

    Sums in 64 bits: the rounded values have to be the same in any order of the sum."""
    c = s["case"]
    nq, _, _, nkb = _geometry(c)
    b, hk, d = c["batch"], c["heads_kv"], c["dim"]
    j = torch.arange(nkb, device="cuda").expand(b, nkb)
    if s["table"] is None:
        page = j + nkb * torch.arange(b, device="cuda")[:, None]
        k = torch.nn.functional.pad(s["k"], (0, 0, 0, 0, 0, nkb * PAGE - c["len"])).reshape(b, nkb, PAGE, hk, d)
    else:
        page = s["table"].long()
        if s["first"] is not None:  # only the blocks from the first new token on: those of nq tokens at most
            width = (nq + PAGE - 2) // PAGE + 1
            j = (s["first"].long()[:, None] // PAGE + torch.arange(width, device="cuda"))
            page = page.gather(1, j.clamp(max=nkb - 1))
        k = s["k"][page]
    kept = (s["lens"].long()[:, None] - j * PAGE).clamp(0, PAGE)
    inside = torch.arange(PAGE, device="cuda") < kept[..., None]
    total = torch.where(inside[..., None, None], k.double(), 0.0).sum(2)
    top = total.abs().amax(-1)
    one = torch.full_like(top, 127.0)
    values = torch.where(top[..., None] > 0, torch.round(total * (one / top)[..., None]), 0.0).to(torch.int8)
    scale = torch.where(top > 0, top / (one * kept[..., None]), 0.0).float()
    live = (kept > 0) & (j < nkb)
    s["pooled"][page[live]] = values[live]
    s["pooled_scale"][page[live]] = scale[live]


def _select(s):
    """The blocks with the highest scores: the queries' sum in 8 bits times the pooled key, and its scale.

    The first block and the queries' own are always among them; ties go to the lower block."""
    c = s["case"]
    nq, q_block, nqb, nkb = _geometry(c)
    b, hk, hq, d = c["batch"], c["heads_kv"], c["heads_q"], c["dim"]
    start, n = s["starts"].long()[:, None], s["lens"].long()[:, None]
    t = torch.arange(nqb * q_block, device="cuda")
    live = (t < nq) & (start + t >= 0) & (start + t < n)
    q = torch.nn.functional.pad(s["q"], (0, 0, 0, 0, 0, nqb * q_block - nq))
    q = torch.where(live[:, :, None, None], q, 0).reshape(b, nqb, q_block, hk, hq // hk, d)
    total = q.double().sum((2, 4))
    top = total.abs().amax(-1, keepdim=True)
    values = torch.where(top > 0, torch.round(total * (torch.full_like(top, 127.0) / top)), 0.0).float()
    if s["table"] is None:
        page = torch.arange(b * nkb, device="cuda").reshape(b, nkb)
    else:
        page = s["table"].long()
    # whole numbers below 2^24: the product is exact in 32 bits
    score = values.permute(0, 2, 1, 3) @ s["pooled"][page].float().permute(0, 2, 3, 1)
    score = score * s["pooled_scale"][page].permute(0, 2, 1)[:, :, None] + 0.0
    last = torch.where(live, start + t, -1).reshape(b, nqb, q_block).amax(-1)
    count = torch.where(last >= 0, last // PAGE + 1, 0)[:, None, :, None]
    j = torch.arange(nkb, device="cuda")
    score = torch.where((j < 1) | (j >= count - 1), math.inf, score)
    score = torch.where(j < count, score, -math.inf)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :c["blocks"]]
    if best.shape[-1] < c["blocks"]:
        best = torch.nn.functional.pad(best, (0, c["blocks"] - best.shape[-1]), value=nkb)
    fits = torch.arange(c["blocks"], device="cuda") < count
    best = torch.where(fits, best, nkb + PAGE).sort(-1).values
    s["lists"] = torch.where(best < nkb, best, -1).to(torch.int32)


def _gathered(s):
    """Queries, keys and values of each list in 32 bits, with what each query sees of them."""
    c = s["case"]
    nq, q_block, nqb, nkb = _geometry(c)
    b, hk, hq, d = c["batch"], c["heads_kv"], c["heads_q"], c["dim"]
    group = hq // hk
    if c["op"] == "cache" and not c["sparse"]:
        blocks = torch.arange(nkb, device="cuda").expand(b, hk, nqb, nkb)
    else:
        blocks = s["lists"].long()
    tok = (blocks.clamp(min=0)[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(-2)
    known = (blocks >= 0).repeat_interleave(PAGE, -1) & (tok < s["lens"].long()[:, None, None, None])
    bi = torch.arange(b, device="cuda")[:, None, None, None]
    hi = torch.arange(hk, device="cuda")[None, :, None, None]
    if s["table"] is None:
        row = tok.clamp(max=c["len"] - 1)
        k, v = s["k"][bi, row, hi].float(), s["v"][bi, row, hi].float()
    else:
        page = s["table"].long()[bi, tok // PAGE]
        k, v = s["k"][page, tok % PAGE, hi].float(), s["v"][page, tok % PAGE, hi].float()
        row = tok

    def rows(x):
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, nqb * q_block - nq))
        return x.reshape(b, nqb, q_block, hk, group, d).permute(0, 3, 1, 2, 4, 5).reshape(b, hk, nqb, -1, d).float()

    t = torch.arange(nqb * q_block, device="cuda").reshape(nqb, q_block)
    pos = s["starts"].long()[:, None, None] + t
    live = (t < nq) & (pos >= 0) & (pos < s["lens"].long()[:, None, None])
    if s["tree"] is not None:
        draft = tok - s["starts"].long()[:, None, None, None]
        bits = torch.nn.functional.pad(s["tree"], (0, nqb * q_block - nq)).reshape(b, 1, nqb, q_block, 1)
        sees = (draft[..., None, :] < 0) | ((bits >> draft.clamp(0, 63)[..., None, :]) & 1).bool()
    else:
        sees = tok[..., None, :] <= pos[:, None, :, :, None]
    sees = (sees & known[..., None, :] & live[:, None, :, :, None]).repeat_interleave(group, -2)
    return rows(s["q"]), k, v, sees, rows, (bi, row, hi)


def _back(s, x):
    """Rows of the lists back in the order of the queries."""
    c = s["case"]
    nq, q_block, nqb, _ = _geometry(c)
    b, hk, hq = c["batch"], c["heads_kv"], c["heads_q"]
    x = x.reshape(b, hk, nqb, q_block, hq // hk, -1).permute(0, 2, 3, 1, 4, 5)
    return x.reshape(b, nqb * q_block, hq, -1)[:, :nq]


def _attend(s):
    q, k, v, sees, rows, where = _gathered(s)
    score = torch.where(sees, (q @ k.transpose(-1, -2)) * s["scale"], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    some = total > 0
    o = torch.where(some, (p @ v) / total, 0.0)
    lse = torch.where(some, top + torch.log(total), -math.inf)
    return o, lse, (q, k, v, rows, where, p, total, some)


def run(state):
    s = state
    c = s["case"]
    if own:
        import sparse_dense_matrix_amd as S
        at = {"lens": s["lens"], "starts": s["starts"]}
        if c["op"] == "select":
            S.spmm_execute_attn_pool(s["plan"], s["k"], s["pooled"], s["pooled_scale"], lens=s["lens"],
                                     table=s["table"], first=s["first"])
            S.spmm_execute_attn_select(s["plan"], s["q"], s["pooled"], s["pooled_scale"], s["lists"],
                                       table=s["table"], **at)
            return {"lists": s["lists"], "pooled": s["pooled"], "scale": s["pooled_scale"]}
        if c["op"] == "cache":
            S.spmm_execute_attn_cache(s["plan"], s["q"], s["k"], s["v"], s["o"], s["lse"], table=s["table"],
                                      lists=s["lists"] if c["sparse"] else None, tree=s["tree"], **at)
            return {"o": s["o"], "lse": s["lse"]}
        S.spmm_execute_attn(s["plan"], s["q"], s["k"], s["v"], s["lists"], s["o"], s["lse"], **at)
        if c["op"] == "forward":
            return {"o": s["o"], "lse": s["lse"]}
        S.spmm_execute_attn_backward(s["plan"], s["grad"], s["q"], s["k"], s["v"], s["lists"], s["o"], s["lse"],
                                     s["dq"], s["dk"], s["dv"], **at)
        return {"o": s["o"], "lse": s["lse"], "dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}
    if c["op"] == "select":
        _pool(s)
        _select(s)
        return {"lists": s["lists"], "pooled": s["pooled"], "scale": s["pooled_scale"]}
    o, lse, (q, k, v, rows, (bi, row, hi), p, total, some) = _attend(s)
    dtype = s["q"].dtype
    out = {"o": _back(s, o).to(dtype), "lse": _back(s, lse)[..., 0].transpose(1, 2).contiguous()}
    if c["op"] != "train":
        return out
    p = torch.where(some, p / total, 0.0)
    do = rows(s["grad"])
    gv = p.transpose(-1, -2) @ do
    ds = p * ((do @ v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)) * s["scale"]
    out["dq"] = _back(s, ds @ k).to(dtype)
    gk = ds.transpose(-1, -2) @ q
    dk, dv = torch.zeros((2,) + tuple(s["k"].shape), dtype=torch.float32, device="cuda")
    at = (bi.expand(row.shape), row, hi.expand(row.shape))
    out["dk"] = dk.index_put_(at, gk, accumulate=True).to(dtype)
    out["dv"] = dv.index_put_(at, gv, accumulate=True).to(dtype)
    return out


# ---- from the definition, in 64 bits ---------------------------------------

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    nq, q_block, nqb, nkb = _geometry(c)
    b, hk, hq, d = c["batch"], c["heads_kv"], c["heads_q"], c["dim"]
    lens = _lens(c)
    dev = s["q"].device
    if c["op"] == "select":  # lists and 8-bit values are whole numbers; the scales are not
        scale = s["pooled_scale"].double()
        for i, n in enumerate(lens):
            for j in range(nkb):
                if j * PAGE >= n:
                    continue
                page = i * nkb + j if s["table"] is None else int(s["table"][i, j])
                x = s["k"][i, j * PAGE:min(n, (j + 1) * PAGE)] if s["table"] is None else s["k"][page, :min(PAGE, n - j * PAGE)]
                scale[page] = x.double().mean(0).abs().amax(-1) / 127
        return {"lists": None, "pooled": None, "scale": scale}
    o = torch.zeros((b, nq, hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((b, hq, nq), -math.inf, dtype=torch.float64, device=dev)
    train = c["op"] == "train"
    if train:
        dq, dk, dv = (torch.zeros(s[x].shape, dtype=torch.float64, device=dev) for x in ("q", "k", "v"))
    for i, n in enumerate(lens):
        start = n - nq if c["tokens"] else 0
        if s["table"] is None:
            ki, vi = s["k"][i, :n].double(), s["v"][i, :n].double()
        else:
            use = s["table"][i, :-(-n // PAGE)].long()
            ki = s["k"][use].reshape(-1, hk, d)[:n].double()
            vi = s["v"][use].reshape(-1, hk, d)[:n].double()
        key = torch.arange(n, device=dev)
        here = min(nq, n - start)
        for h in range(hk):
            chosen = None
            if c["op"] != "cache" or c["sparse"]:
                chosen = torch.zeros((nqb, nkb + 1), dtype=torch.bool, device=dev)
                ids = s["lists"][i, h].long()
                chosen.scatter_(1, torch.where(ids >= 0, ids, nkb), True)
                chosen[:, nkb] = False
            for lo in range(0, here, 8192):
                t = torch.arange(lo, min(lo + 8192, here), device=dev)
                if s["tree"] is not None:
                    draft = key[None] - start
                    m = (draft < 0) | ((s["tree"][i][t][:, None] >> draft.clamp(0, 63)) & 1).bool()
                else:
                    m = key[None] <= start + t[:, None]
                if chosen is not None:
                    m = m & chosen[t // q_block][:, key // PAGE]
                for g in range(h * (hq // hk), (h + 1) * (hq // hk)):
                    qh = s["q"][i, t, g].double()
                    z = (qh @ ki[:, h].T / math.sqrt(d)).masked_fill_(~m, -math.inf)
                    e = torch.logsumexp(z, -1)
                    w = torch.exp_(z.sub_(torch.where(torch.isinf(e), 0.0, e)[:, None]))
                    o[i, t, g] = w @ vi[:, h]
                    lse[i, g, t] = e
                    if train:
                        go = s["grad"][i, t, g].double()
                        dv[i, :n, h] += w.T @ go
                        dz = go @ vi[:, h].T
                        dz.sub_((go * o[i, t, g]).sum(-1, keepdim=True)).mul_(w).div_(math.sqrt(d))
                        dq[i, t, g] = dz @ ki[:, h]
                        dk[i, :n, h] += dz.T @ qh
    out = {"o": o, "lse": lse}
    if train:
        out.update(dq=dq, dk=dk, dv=dv)
    return out
