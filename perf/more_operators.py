"""Cases for timing what stands around attention over a cache: norms and
position rotation of queries and keys (forward, and forward with the
gradients), a cache in 8 bits as it is written, read back and pooled, and
attention of new or drafted tokens over it.

A cache holds pages of 64 keys reached through a table.  Each token's key and
value of each head stand as 8-bit codes with a scale: top = max|x| of the row,
scale = top / 127, code = round(127 x / top).  Token t of a sequence stands at
position start + t; it counts when that is in [0, len).
"""
import math

import torch

own = False

PAGE = 64
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---- cases -----------------------------------------------------------------

def _case(name, op, **kw):
    c = {"op": op, "batch": 1, "len": 0, "tokens": 0, "heads_q": 32, "heads_kv": 8, "dim": 128, "dtype": "bf16",
         "ragged": False, "axes": 1, "pairs": 0, "interleaved": False, "norm": True, "tree": False, "blocks": 0}
    c.update(kw)
    c["pairs"] = c["pairs"] or c["dim"] // 2
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a decode step: the new token of 32 ragged sequences, far positions
        _case("rope step 32", "rope", batch=32, len=32768, tokens=1, ragged=True),
        # images: time, height and width turn 16 channels each, neighbours in pairs, 16 channels stay
        _case("rope image ragged 3x777", "rope", batch=3, len=777, tokens=777, heads_q=6, heads_kv=2, dim=64,
              dtype="f16", ragged=True, axes=3, pairs=24, interleaved=True),
        # training on a long text: forward, gradients of q, k and both norms' weights
        _case("rope train 16k", "rope train", len=16384, tokens=16384),
        # a decode step writes one token of each of 32 sequences
        _case("write step 32", "write", batch=32, len=16384, tokens=1, ragged=True),
        # a prompt goes to its pages
        _case("write prompt 16k", "write", len=16384, tokens=16384),
        # a decode step pools the page that its new token stands in
        _case("pool step 32", "pool", batch=32, len=16384, tokens=1, ragged=True),
        # all pages of ragged prompts
        _case("pool 4x8k", "pool", batch=4, len=8191, tokens=8191, ragged=True),
        # a short ragged prefix read back for the next prompt
        _case("read ragged 3x777", "read", batch=3, len=777, heads_q=6, heads_kv=2, dim=64, dtype="f16", ragged=True),
        # a long prefix read back
        _case("read 32k", "read", len=32768),
        # one user's next token: latency counts
        _case("cache step 1x4097", "cache", len=4097, tokens=1),
        # a full batch of long ragged sequences
        _case("cache step 32x32k", "cache", batch=32, len=32768, tokens=1, ragged=True),
        # 24 drafted tokens of a tree, checked at once
        _case("cache tree 16x8k", "cache", batch=16, len=8192, tokens=24, ragged=True, tree=True, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope train", "write", "pool", "read", "cache", "cache"])
    dim, kv = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8])
    hq = kv * min(rng.choice([1, 2, 3, 4, 5, 8, 16]), 64 // kv)
    kw = {"heads_q": hq, "heads_kv": kv, "dim": dim, "dtype": rng.choice(["bf16", "bf16", "f16"]),
          "ragged": rng.random() < 0.5}
    step = op != "rope train" and rng.random() < 0.5
    if op == "cache":
        kind = rng.choice(["step", "step", "tree", "chosen", "chunk"])
        batch = _log(rng, 1, 48 if kind != "chunk" else 4)
        tokens = {"step": 1, "tree": rng.randint(2, 64), "chosen": rng.choice([1, rng.randint(2, 12)]),
                  "chunk": rng.randint(65, 400)}[kind]
        length = max(tokens, _log(rng, 1, min(32768 if kind != "chunk" else 8192, 700000 // batch)))
        return _case(None, op, batch=batch, len=length, tokens=tokens, tree=kind == "tree",
                     blocks=rng.randint(2, 48) if kind == "chosen" else 0, **kw)
    batch = _log(rng, 1, 48 if step else 4)
    length = _log(rng, 1, min(32768, 300000 // batch) if step else 16384 // batch)
    tokens = min(length, rng.choice([1, 1, rng.randint(2, 64)])) if step and op != "read" else length
    if op in ("rope", "rope train"):
        kw["pairs"] = 8 * rng.randint(1, dim // 16)
        kw["interleaved"] = rng.random() < 0.4
        kw["axes"] = rng.choice([1, 1, 2, 3])
        kw["norm"] = rng.random() < 0.8
    return _case(None, op, batch=batch, len=length, tokens=0 if op == "read" else tokens, **kw)


def _lens(c):
    """Lengths of the sequences: they differ where the case is ragged."""
    least = max(1, min(c["tokens"], 64))
    return [max(least, c["len"] - (i * 2654435761 % 997) * c["len"] // 1300 if c["ragged"] else c["len"])
            for i in range(c["batch"])]


def _starts(c):
    """Positions of the first tokens: the last `tokens` of a sequence are new, or all of it is."""
    return [0 if c["tokens"] == c["len"] else max(0, n - c["tokens"]) for n in _lens(c)]


def _blocks(c):
    return -(-c["len"] // PAGE)


def work(case):
    c, d, hq, hk, elem = case, case["dim"], case["heads_q"], case["heads_kv"], 2
    lens, starts = _lens(c), _starts(c)
    new = sum(min(c["tokens"], n - s) for n, s in zip(lens, starts))
    if c["op"] in ("rope", "rope train"):
        rows, train = new * (hq + hk), c["op"] == "rope train"
        place = new * 4 * c["axes"] if c["axes"] > 1 else 0
        weights = 2 * d * 4 * (2 if train else 1) if c["norm"] else 0
        return {"bytes": float(rows * d * elem * (4 if train else 2) + place + weights),
                "flops": float(rows * d * (20 if train else 8))}
    if c["op"] == "write":
        return {"bytes": float(2 * new * hk * (d * (elem + 1) + 4)), "flops": float(2 * new * hk * d * 3)}
    if c["op"] == "read":
        return {"bytes": float(2 * sum(lens) * hk * (d * (elem + 1) + 4)), "flops": float(2 * sum(lens) * hk * d)}
    if c["op"] == "pool":
        blocks = sum(-(-n // PAGE) - s // PAGE for n, s in zip(lens, starts))
        keys = sum(n - s // PAGE * PAGE for n, s in zip(lens, starts))
        return {"bytes": float((keys + blocks) * hk * (d + 4)), "flops": float(2 * keys * hk * d)}
    t = c["tokens"]
    read = [min(n, c["blocks"] * PAGE) if c["blocks"] else n for n in lens]
    pairs = sum(t * max(0, n - t) + min(t, n) * (min(t, n) + 1) // 2 for n in read)
    return {"bytes": float(2 * sum(read) * hk * (d + 4) + c["batch"] * t * hq * (2 * d * elem + 4)),
            "flops": float(4 * d * hq * pairs)}


# ---- inputs ----------------------------------------------------------------

def _quantised(x):
    """8-bit codes of rows, and their scales.

    In 64 bits: a value next to the border of two codes keeps its side."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    code = torch.where(top > 0, torch.round(127.0 * x / torch.where(top > 0, top, 1.0)), 0.0).to(torch.int8)
    return code, (top[..., 0] / 127.0).float()


def _cache(s, g):
    """Pages of keys with strong channels and a topic, and of values of uneven size, in 8 bits."""
    c = s["case"]
    hk, d, pages = c["heads_kv"], c["dim"], c["batch"] * _blocks(c)
    s["table"] = torch.randperm(pages, generator=g, device="cuda").reshape(c["batch"], -1).to(torch.int32)
    s["k8"], s["v8"] = torch.empty((2, pages, PAGE, hk, d), dtype=torch.int8, device="cuda")
    s["k_scale"], s["v_scale"] = torch.empty((2, pages, hk, PAGE), dtype=torch.float32, device="cuda")
    channel = torch.exp(0.5 * torch.randn((hk, d), generator=g, device="cuda"))
    topics = 0.5 * torch.randn((16, 1, hk, d), generator=g, device="cuda")
    for lo in range(0, pages, 1024):
        n = min(1024, pages - lo)
        k = torch.randn((n, PAGE, hk, d), generator=g, device="cuda") * channel
        k = k + topics[torch.randint(0, 16, (n,), generator=g, device="cuda")]
        v = torch.randn((n, PAGE, hk, d), generator=g, device="cuda")
        v = v * torch.exp(0.5 * torch.randn((n, PAGE, hk, 1), generator=g, device="cuda"))
        for x, code, scale in ((k, "k8", "k_scale"), (v, "v8", "v_scale")):
            x = _quantised(x.to(DTYPES[c["dtype"]]))
            s[code][lo:lo + n], s[scale][lo:lo + n] = x[0], x[1].transpose(1, 2)
    return topics


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype, d, hq, hk, b, n = DTYPES[c["dtype"]], c["dim"], c["heads_q"], c["heads_kv"], c["batch"], c["tokens"]
    s = {"case": c, "lens": torch.tensor(_lens(c), dtype=torch.int32, device="cuda"),
         "starts": torch.tensor(_starts(c), dtype=torch.int32, device="cuda")}

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if c["op"] in ("rope", "rope train"):
        # projections: channels of uneven size, heads side by side in one buffer
        channel = torch.exp(0.7 * normal(hq + hk, d))
        s["qk"] = (normal(b, n, hq + hk, d) * channel).to(dtype)
        s["q_weight"], s["k_weight"] = (1.0 + 0.2 * normal(2, d)) if c["norm"] else (None, None)
        s["freqs"] = [10000.0 ** (-p / c["pairs"]) for p in range(c["pairs"])]
        s["axis"] = [p * c["axes"] // c["pairs"] for p in range(c["pairs"])]
        s["positions"] = None
        if c["axes"] > 1:  # frames of 24 x 32 patches after the text
            t = s["starts"].long()[:, None] + torch.arange(n, device="cuda")
            s["positions"] = torch.stack((t // 768, t // 32 % 24, t % 32)[:c["axes"]]).to(torch.int32).contiguous()
        if c["op"] == "rope train":
            s["q_grad"], s["k_grad"] = normal(b, n, hq, d).to(dtype), normal(b, n, hk, d).to(dtype)
        s["q_out"], s["k_out"] = s["qk"].new_zeros((b, n, hq, d)), s["qk"].new_zeros((b, n, hk, d))
    elif c["op"] == "read":
        _cache(s, g)
        s["k"], s["v"] = torch.zeros((2, b, c["len"], hk, d), dtype=dtype, device="cuda")
    else:
        topics = _cache(s, g)
    if c["op"] == "write":
        s["k"], s["v"] = normal(b, n, hk, d).to(dtype), normal(b, n, hk, d).to(dtype)
    if c["op"] == "pool":
        s["first"] = s["starts"]  # the pages before the new tokens are pooled already
        s["pooled"] = torch.zeros((b * _blocks(c), hk, d), dtype=torch.int8, device="cuda")
        s["pooled_scale"] = torch.zeros((b * _blocks(c), hk), dtype=torch.float32, device="cuda")
    if c["op"] == "cache":
        part = topics[torch.randint(0, 16, (b,), generator=g, device="cuda")].repeat_interleave(hq // hk, dim=2)
        s["q"] = (normal(b, n, hq, d) + part).to(dtype)
        s["tree"] = s["lists"] = None
        if c["tree"]:  # each drafted token hangs below an earlier one, or below the text
            parent = (torch.rand((b, n), generator=g, device="cuda") * torch.arange(n, device="cuda")).long()
            bits = torch.zeros((b, n), dtype=torch.int64, device="cuda")
            bits[:, 0] = 1
            for t in range(1, n):
                bits[:, t] = bits.gather(1, parent[:, t:t + 1])[:, 0] | (1 << t if t < 63 else -(1 << 63))
            s["tree"] = bits
        if c["blocks"]:  # a choice made before: some of the sequence's blocks, the last one among them
            last = (s["lens"].long() - 1)[:, None] // PAGE
            score = torch.rand((b, hk, _blocks(c)), generator=g, device="cuda")
            j = torch.arange(_blocks(c), device="cuda")
            score = torch.where(j == last[:, None], 2.0, torch.where(j < last[:, None], score, -1.0))
            best = score.sort(dim=-1, descending=True)
            ids = torch.where(best.values >= 0, best.indices, _blocks(c))[..., :c["blocks"]]
            ids = torch.nn.functional.pad(ids, (0, c["blocks"] - ids.shape[-1]), value=_blocks(c)).sort(-1).values
            s["lists"] = torch.where(ids < _blocks(c), ids, -1).to(torch.int32)[:, :, None].contiguous()
    if own:  # the plan and the buffers that a program keeps
        import sparse_dense_matrix_amd as S
        kind = {"bf16": S.BF16, "f16": S.F16}[c["dtype"]]
        if c["op"] in ("rope", "rope train"):
            s["plan"] = S.spmm_plan_attn_rope(b, n, hq, hk, d, s["freqs"], axis=s["axis"], dtype=kind,
                                              interleaved=c["interleaved"], eps=EPS, backward=c["op"] == "rope train")
            if c["op"] == "rope train":
                s["dq"], s["dk"] = torch.empty_like(s["q_out"]), torch.empty_like(s["k_out"])
                s["dq_weight"], s["dk_weight"] = torch.empty((2, d), device="cuda") if c["norm"] else (None, None)
        else:
            s["plan"] = S.spmm_plan_attn(b, max(1, n), _blocks(c) * PAGE if c["op"] != "read" else c["len"], hq, hk, d,
                                         dtype=kind, max_blocks=c["blocks"] or 16)
        if c["op"] == "cache":
            s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty((b, hq, n), dtype=torch.float32, device="cuda")
    return s


# ---- plain forms -----------------------------------------------------------

def _live(s, tokens):
    pos = s["starts"].long()[:, None] + torch.arange(tokens, device="cuda")
    return pos, (pos >= 0) & (pos < s["lens"].long()[:, None])


def _angles(s):
    """cos and sin [b, tokens, 1, pairs]; the angles of far positions in 64 bits."""
    c = s["case"]
    place = _live(s, c["tokens"])[0].expand(c["axes"], -1, -1) if s["positions"] is None else s["positions"].long()
    freqs = torch.tensor(s["freqs"], dtype=torch.float64, device="cuda")
    angle = (place[torch.tensor(s["axis"], device="cuda")].permute(1, 2, 0) * freqs)[:, :, None]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turn(c, x, cos, sin):
    """Pairs of channels turned by their angles; the channels after them stay."""
    n = c["pairs"]
    if c["interleaved"]:
        u, v = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack((u * cos - v * sin, u * sin + v * cos), -1).flatten(-2)
    else:
        u, v = x[..., :n], x[..., n:2 * n]
        y = torch.cat((u * cos - v * sin, u * sin + v * cos), -1)
    return torch.cat((y, x[..., 2 * n:]), -1)


def _rope(s):
    c = s["case"]
    live = _live(s, c["tokens"])[1][..., None, None]
    cos, sin = _angles(s)
    q, k = s["qk"].split((c["heads_q"], c["heads_kv"]), 2)
    out = {}
    for name, x, w in (("q", q, s["q_weight"]), ("k", k, s["k_weight"])):
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        y = _turn(c, x if w is None else x * r * w, cos, sin)
        out[name] = torch.where(live, y, s[name + "_out"].float()).to(s["qk"].dtype)
        if c["op"] == "rope train":
            dy = _turn(c, torch.where(live, s[name + "_grad"].float(), 0.0), cos, -sin)
            dx = dy
            if w is not None:
                out["d" + name + "_weight"] = (dy * torch.where(live, x * r, 0.0)).sum((0, 1, 2))
                wdy = dy * w
                dx = r * wdy - x * r * r * r * (wdy * x).mean(-1, keepdim=True)
            out["d" + name] = torch.where(live, dx, 0.0).to(s["qk"].dtype)
    return out


def _write(s):
    pos, live = _live(s, s["case"]["tokens"])
    page = s["table"].long().gather(1, torch.where(live, pos, 0) // PAGE)[live]
    at = pos[live] % PAGE
    for x, code, scale in (("k", "k8", "k_scale"), ("v", "v8", "v_scale")):
        codes, scales = _quantised(s[x][live])
        s[code][page, at] = codes
        s[scale][page, :, at] = scales
    return {x: s[x] for x in ("k8", "v8", "k_scale", "v_scale")}


def _values(s, code, scale, page):
    """What the codes of pages stand for, [..., 64, heads, dim] in 32 bits."""
    return s[code][page].float() * s[scale][page].transpose(-1, -2)[..., None]


def _read(s):
    c = s["case"]
    inside = (torch.arange(c["len"], device="cuda") < s["lens"].long()[:, None])[..., None, None]
    out = {}
    for x, code, scale in (("k", "k8", "k_scale"), ("v", "v8", "v_scale")):
        y = _values(s, code, scale, s["table"].long()).flatten(1, 2)[:, :c["len"]]
        out[x] = torch.where(inside, y, s[x].float()).to(s[x].dtype)
    return out


def _pool(s):
    """Mean keys in 8 bits with a scale, of the blocks from the first new token on; sums in 64 bits."""
    c = s["case"]
    width = min(_blocks(c), (c["tokens"] + PAGE - 2) // PAGE + 1)
    j = s["first"].long()[:, None] // PAGE + torch.arange(width, device="cuda")
    page = s["table"].long().gather(1, j.clamp(max=_blocks(c) - 1))
    kept = (s["lens"].long()[:, None] - j * PAGE).clamp(0, PAGE)
    inside = (torch.arange(PAGE, device="cuda") < kept[..., None])[..., None, None]
    k = s["k8"][page].double() * s["k_scale"][page].double().transpose(-1, -2)[..., None]
    total = torch.where(inside, k, 0.0).sum(2)
    top = total.abs().amax(-1)
    some = top > 0
    values = torch.where(some[..., None], torch.round(total * (127.0 / torch.where(some, top, 1.0))[..., None]), 0.0)
    live = (kept > 0) & (j < _blocks(c))
    s["pooled"][page[live]] = values.to(torch.int8)[live]
    s["pooled_scale"][page[live]] = (top / (127.0 * kept.clamp(min=1)[..., None])).float()[live]
    return {"pooled": s["pooled"], "pooled_scale": s["pooled_scale"]}


def _attend(s):
    c = s["case"]
    b, n, hk, hq, d = c["batch"], c["tokens"], c["heads_kv"], c["heads_q"], c["dim"]
    if c["blocks"]:
        block = s["lists"][:, :, 0].long()
        page = s["table"].long()[:, None].expand(-1, hk, -1).gather(2, block.clamp(min=0))
        h = torch.arange(hk, device="cuda")[:, None]
        k = (s["k8"][page, :, h].float() * s["k_scale"][page, h][..., None]).flatten(2, 3)
        v = (s["v8"][page, :, h].float() * s["v_scale"][page, h][..., None]).flatten(2, 3)
        key = (block.clamp(min=0)[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(-2)
        known = (block >= 0).repeat_interleave(PAGE, -1)
    else:
        k = _values(s, "k8", "k_scale", s["table"].long()).flatten(1, 2).transpose(1, 2)
        v = _values(s, "v8", "v_scale", s["table"].long()).flatten(1, 2).transpose(1, 2)
        key = torch.arange(_blocks(c) * PAGE, device="cuda").expand(b, 1, -1)
        known = torch.ones_like(key, dtype=torch.bool)
    pos, live = _live(s, n)
    if c["tree"]:
        draft = (key - s["starts"].long()[:, None, None])[:, :, None]
        sees = (draft < 0) | ((s["tree"][:, None, :, None] >> draft.clamp(0, 63)) & 1).bool()
    else:
        sees = key[:, :, None] <= pos[:, None, :, None]
    sees = sees & (known & (key < s["lens"].long()[:, None, None]))[:, :, None] & live[:, None, :, None]
    sees = sees.repeat_interleave(hq // hk, 2)
    q = s["q"].float().reshape(b, n, hk, -1, d).transpose(1, 2).reshape(b, hk, -1, d)
    score = torch.where(sees, (q @ k.transpose(-1, -2)) / math.sqrt(d), -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    some = total > 0
    o = torch.where(some, (p @ v) / total, 0.0).reshape(b, hk, n, -1, d).transpose(1, 2).reshape(b, n, hq, d)
    lse = torch.where(some, top + torch.log(total), -math.inf).reshape(b, hk, n, -1).transpose(2, 3).reshape(b, hq, n)
    return {"o": o.to(s["q"].dtype), "lse": lse.contiguous()}


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"rope": _rope, "rope train": _rope, "write": _write, "read": _read, "pool": _pool,
                "cache": _attend}[c["op"]](s)
    import sparse_dense_matrix_amd as S
    at = {"lens": s["lens"], "starts": s["starts"]}
    if c["op"] in ("rope", "rope train"):
        q, k = s["qk"].split((c["heads_q"], c["heads_kv"]), 2)
        at.update(q_weight=s["q_weight"], k_weight=s["k_weight"], positions=s["positions"])
        S.spmm_execute_attn_rope(s["plan"], q, k, s["q_out"], s["k_out"], **at)
        out = {"q": s["q_out"], "k": s["k_out"]}
        if c["op"] == "rope train":
            S.spmm_execute_attn_rope_backward(s["plan"], s["q_grad"], s["k_grad"], q, k, s["dq"], s["dk"],
                                              dq_weight=s["dq_weight"], dk_weight=s["dk_weight"], **at)
            out.update(dq=s["dq"], dk=s["dk"])
            if c["norm"]:
                out.update(dq_weight=s["dq_weight"], dk_weight=s["dk_weight"])
        return out
    cache = (s["k8"], s["v8"], s["k_scale"], s["v_scale"])
    if c["op"] == "write":
        S.spmm_execute_attn_write(s["plan"], s["k"], s["v"], *cache, table=s["table"], **at)
        return {x: s[x] for x in ("k8", "v8", "k_scale", "v_scale")}
    if c["op"] == "read":
        S.spmm_execute_attn_read(s["plan"], *cache, s["k"], s["v"], table=s["table"], lens=s["lens"])
        return {"k": s["k"], "v": s["v"]}
    if c["op"] == "pool":
        S.spmm_execute_attn_pool8(s["plan"], s["k8"], s["k_scale"], s["pooled"], s["pooled_scale"], table=s["table"],
                                  lens=s["lens"], first=s["first"])
        return {"pooled": s["pooled"], "pooled_scale": s["pooled_scale"]}
    S.spmm_execute_attn_cache8(s["plan"], s["q"], *cache, s["o"], s["lse"], table=s["table"], lists=s["lists"],
                               tree=s["tree"], **at)
    return {"o": s["o"], "lse": s["lse"]}


# ---- from the definition, in 64 bits ---------------------------------------

def _exact_rope(s):
    """Turning as a product of complex numbers, gradients by differentiation."""
    c = s["case"]
    n, train = c["tokens"], c["op"] == "rope train"
    freqs = torch.tensor(s["freqs"], dtype=torch.float64, device="cuda")
    angle = torch.zeros((c["batch"], n, 1, c["pairs"]), dtype=torch.float64, device="cuda")
    live = torch.zeros((c["batch"], n, 1, 1), dtype=torch.bool, device="cuda")
    for i, (length, start) in enumerate(zip(_lens(c), _starts(c))):
        t = start + torch.arange(n, device="cuda")
        live[i, :, 0, 0] = (t >= 0) & (t < length)
        for p in range(c["pairs"]):
            at = t if s["positions"] is None else s["positions"][s["axis"][p], i]
            angle[i, :, 0, p] = at.double() * freqs[p]
    turn = torch.polar(torch.ones_like(angle), angle)
    out = {}
    q, k = s["qk"].split((c["heads_q"], c["heads_kv"]), 2)
    for name, x, w in (("q", q, s["q_weight"]), ("k", k, s["k_weight"])):
        x = x.double().requires_grad_(train)
        w = None if w is None else w.double().requires_grad_(train)
        y = x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + EPS).sqrt() * w
        head, rest = y[..., :2 * c["pairs"]], y[..., 2 * c["pairs"]:]
        if c["interleaved"]:
            head = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * turn).flatten(-2)
        else:
            head = torch.complex(*head.chunk(2, -1)) * turn
            head = torch.cat((head.real, head.imag), -1)
        y = torch.cat((head, rest), -1)
        out[name] = torch.where(live, y, 0.0).detach()
        if train:
            grad = torch.where(live, s[name + "_grad"].double(), 0.0)
            found = torch.autograd.grad(y, [x] if w is None else [x, w], grad)
            out["d" + name] = found[0]
            if w is not None:
                out["d" + name + "_weight"] = found[1]
    return out


def _exact_pages(s, code, scale, i, n):
    """Keys or values 0 .. n - 1 of sequence i, [n, heads, dim]."""
    use = s["table"][i, :-(-n // PAGE)].long()
    x = s[code][use].double() * s[scale][use].double().transpose(1, 2)[..., None]
    return x.reshape(-1, *x.shape[2:])[:n]


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    lens, starts = _lens(c), _starts(c)
    hk, group, d = c["heads_kv"], c["heads_q"] // c["heads_kv"], c["dim"]
    if c["op"] in ("rope", "rope train"):
        return _exact_rope(s)
    if c["op"] == "write":  # codes are whole numbers; scales are not
        out = {"k8": None, "v8": None, "k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double()}
        for i, (n, start) in enumerate(zip(lens, starts)):
            at = torch.arange(start, min(n, start + c["tokens"]), device="cuda")
            page = s["table"][i].long()[at // PAGE]
            for x, scale in (("k", "k_scale"), ("v", "v_scale")):
                out[scale][page, :, at % PAGE] = s[x][i, :len(at)].double().abs().max(-1).values / 127
        return out
    if c["op"] == "read":
        out = {x: torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in ("k", "v")}
        for i, n in enumerate(lens):
            out["k"][i, :n] = _exact_pages(s, "k8", "k_scale", i, n)
            out["v"][i, :n] = _exact_pages(s, "v8", "v_scale", i, n)
        return out
    if c["op"] == "pool":
        scale = s["pooled_scale"].double()
        for i, (n, start) in enumerate(zip(lens, starts)):
            k = _exact_pages(s, "k8", "k_scale", i, n)
            for j in range(start // PAGE, -(-n // PAGE)):
                scale[s["table"][i, j]] = k[j * PAGE:(j + 1) * PAGE].mean(0).abs().amax(-1) / 127
        return {"pooled": None, "pooled_scale": scale}
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], c["heads_q"], c["tokens"]), -math.inf, dtype=torch.float64, device="cuda")
    for i, (n, start) in enumerate(zip(lens, starts)):
        k, v = _exact_pages(s, "k8", "k_scale", i, n), _exact_pages(s, "v8", "v_scale", i, n)
        key = torch.arange(n, device="cuda")
        t = torch.arange(min(c["tokens"], n - start), device="cuda")
        if c["tree"]:
            draft = key[None] - start
            m = (draft < 0) | ((s["tree"][i][t][:, None] >> draft.clamp(0, 63)) & 1).bool()
        else:
            m = key[None] <= start + t[:, None]
        for h in range(c["heads_q"]):
            mh = m
            if c["blocks"]:
                chosen = torch.zeros(_blocks(c) + 1, dtype=torch.bool, device="cuda")
                chosen[s["lists"][i, h // group, 0].long()] = True  # -1: the last place, which no key has
                mh = m & chosen[key // PAGE]
            z = (s["q"][i, t, h].double() @ k[:, h // group].T / math.sqrt(d)).masked_fill(~mh, -math.inf)
            e = torch.logsumexp(z, -1)
            o[i, t, h] = torch.exp(z - torch.where(torch.isinf(e), 0.0, e)[:, None]) @ v[:, h // group]
            lse[i, h, t] = e
    return {"o": o, "lse": lse}
