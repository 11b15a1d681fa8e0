"""Block-sparse attention as a model layer uses it, on one GPU: a training
step, a prompt, decode steps over a cache of pages, and a check of drafted
tokens.  Random inputs; every stage is compared with plain attention over the
same blocks.

    python examples/block_sparse_attention.py [--tokens 2000] [--steps 70]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_dense_matrix_amd as S  # noqa: E402

PAGE = 64


class BlockSparseAttention:
    """One layer's attention: 16 query heads over 4 key heads, each block of
    64 queries (each new token, when decoding) reads `blocks` blocks of 64 keys."""

    def __init__(self, batch, tokens, room, blocks=8, heads_q=16, heads_kv=4, dim=128):
        self.batch, self.tokens, self.room = batch, tokens, room
        self.hq, self.hk, self.dim, self.blocks = heads_q, heads_kv, dim, blocks
        pages = -(-room // PAGE)
        shape = (batch, tokens, tokens, heads_q, heads_kv, dim)
        self.train_plan = S.spmm_plan_attn(*shape, max_blocks=blocks, backward=True)
        self.step_plan = S.spmm_plan_attn(batch, 1, pages * PAGE, heads_q, heads_kv, dim, max_blocks=blocks)
        # the cache: pages in any order, reached through a table
        self.table = torch.randperm(batch * pages).reshape(batch, pages).int().cuda()
        self.k, self.v = torch.zeros((2, batch * pages, PAGE, heads_kv, dim), dtype=torch.bfloat16, device="cuda")
        self.pooled = torch.zeros((batch * pages, heads_kv, dim), dtype=torch.int8, device="cuda")
        self.scale = torch.zeros((batch * pages, heads_kv), device="cuda")

    def forward(self, q, k, v):
        """Attention over the prompt's chosen blocks: o, and what backward needs."""
        nkb = -(-self.tokens // PAGE)
        pooled = torch.empty((self.batch * nkb, self.hk, self.dim), dtype=torch.int8, device="cuda")
        scale = torch.empty((self.batch * nkb, self.hk), device="cuda")
        lists = torch.empty((self.batch, self.hk, nkb, self.blocks), dtype=torch.int32, device="cuda")
        o, lse = torch.empty_like(q), torch.empty((self.batch, self.hq, self.tokens), device="cuda")
        S.spmm_execute_attn_pool(self.train_plan, k, pooled, scale)
        S.spmm_execute_attn_select(self.train_plan, q, pooled, scale, lists)
        S.spmm_execute_attn(self.train_plan, q, k, v, lists, o, lse)
        return o, (q, k, v, lists, o, lse)

    def backward(self, grad, saved):
        q, k, v, lists, o, lse = saved
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        S.spmm_execute_attn_backward(self.train_plan, grad, q, k, v, lists, o, lse, dq, dk, dv)
        return dq, dk, dv

    def append(self, k, v, at):
        """New keys and values from position `at` on go to their pages."""
        pos = at + torch.arange(k.shape[1], device="cuda")
        page = self.table[:, pos // PAGE].long()
        self.k[page, pos % PAGE] = k
        self.v[page, pos % PAGE] = v

    def attend(self, q, at, plan, tree=None, choose=True):
        """Queries at positions `at` on over the cache, which holds them already."""
        nq = q.shape[1]
        starts = torch.full((self.batch,), at, dtype=torch.int32, device="cuda")
        lens = starts + nq
        lists = None
        if choose:
            lists = torch.empty((self.batch, self.hk, 1, self.blocks), dtype=torch.int32, device="cuda")
            S.spmm_execute_attn_pool(plan, self.k, self.pooled, self.scale, lens=lens, table=self.table, first=starts)
            S.spmm_execute_attn_select(plan, q, self.pooled, self.scale, lists, lens=lens, starts=starts,
                                       table=self.table)
        o, lse = torch.empty_like(q), torch.empty((self.batch, self.hq, nq), device="cuda")
        S.spmm_execute_attn_cache(plan, q, self.k, self.v, o, lse, table=self.table, lists=lists, tree=tree,
                                  lens=lens, starts=starts)
        return o, lists

    def plain(self, q, k, v, sees):
        """The same in 32 bits over all keys, masked: sees is [batch, heads_kv, queries, keys]."""
        g = self.hq // self.hk
        qt = q.float().transpose(1, 2)
        kt, vt = (x.float().transpose(1, 2).repeat_interleave(g, 1) for x in (k, v))
        s = (qt @ kt.transpose(-1, -2) / math.sqrt(self.dim)).masked_fill(~sees.repeat_interleave(g, 1), -math.inf)
        return (torch.softmax(s, -1) @ vt).transpose(1, 2)


def listed(lists, keys):
    """[batch, heads, lists, keys]: the keys of each list's blocks."""
    hit = torch.zeros((*lists.shape[:3], -(-keys // PAGE) + 1), dtype=torch.bool, device=lists.device)
    hit.scatter_(-1, torch.where(lists >= 0, lists, hit.shape[-1] - 1).long(), True)
    return hit[..., :-1].repeat_interleave(PAGE, -1)[..., :keys]


def near(name, got, want):
    off = ((got.float() - want).norm() / want.norm()).item()
    print(f"{name}: off by {off:.1e} of the norm", flush=True)
    assert off < 2.0 ** -7, name  # a few roundings to bf16


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2000)
    ap.add_argument("--steps", type=int, default=70, help="decode steps")
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    batch, n = 2, a.tokens
    layer = BlockSparseAttention(batch, n, n + a.steps + 64)

    def make(tokens, heads):
        return torch.randn((batch, tokens, heads, layer.dim), device="cuda").bfloat16()

    # a training step
    q, k, v, grad = make(n, layer.hq), make(n, layer.hk), make(n, layer.hk), make(n, layer.hq)
    o, saved = layer.forward(q, k, v)
    dq, dk, dv = layer.backward(grad, saved)
    sees = listed(saved[3], n).repeat_interleave(PAGE, 2)[:, :, :n].tril()
    leaves = [x.float().requires_grad_() for x in (q, k, v)]
    want = layer.plain(*leaves, sees)
    near("prompt", o, want.detach())
    for name, got, w in zip(("dq", "dk", "dv"), (dq, dk, dv), torch.autograd.grad(want, leaves, grad.float())):
        near(name, got, w)

    # decode steps: the prompt's keys go to pages, then one token after another
    layer.append(k, v, 0)
    first = torch.zeros((batch,), dtype=torch.int32, device="cuda")
    pool_plan = S.spmm_plan_attn(batch, n, layer.table.shape[1] * PAGE, layer.hq, layer.hk, layer.dim,
                                 max_blocks=layer.blocks)
    S.spmm_execute_attn_pool(pool_plan, layer.k, layer.pooled, layer.scale, table=layer.table,
                             lens=first + n, first=first)
    for step in range(a.steps):
        q1, k1, v1 = make(1, layer.hq), make(1, layer.hk), make(1, layer.hk)
        layer.append(k1, v1, n + step)
        k, v = torch.cat((k, k1), 1), torch.cat((v, v1), 1)
        o, lists = layer.attend(q1, n + step, layer.step_plan)
    near("decode step %d" % a.steps, o, layer.plain(q1, k, v, listed(lists, k.shape[1])))

    # drafted tokens: 1 and 2 follow 0, 3 follows 1; every page is read
    drafted, at = 4, k.shape[1]
    tree = torch.tensor([0b0001, 0b0011, 0b0101, 0b1011]).expand(batch, drafted).contiguous().cuda()
    q4, k4, v4 = make(drafted, layer.hq), make(drafted, layer.hk), make(drafted, layer.hk)
    layer.append(k4, v4, at)
    k, v = torch.cat((k, k4), 1), torch.cat((v, v4), 1)
    plan = S.spmm_plan_attn(batch, drafted, layer.table.shape[1] * PAGE, layer.hq, layer.hk, layer.dim,
                            max_blocks=layer.blocks)
    o, _ = layer.attend(q4, at, plan, tree=tree, choose=False)
    sees = torch.ones((batch, layer.hk, drafted, at + drafted), dtype=torch.bool, device="cuda")
    sees[..., at:] = (tree[:, None, :, None] >> torch.arange(drafted, device="cuda") & 1).bool()
    near("drafted tokens", o, layer.plain(q4, k, v, sees))


if __name__ == "__main__":
    main()
