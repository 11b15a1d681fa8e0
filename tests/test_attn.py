"""Attention on the CPU: the rules the kernels share with the host, the plan's
decisions, the refusals of every call (tests/attn_driver.cpp drives the
library without a device), and the reference that the GPU tests use, whose
gradients are checked against differences of its forward form."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import attn_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBDIR = os.path.join(ROOT, "sparse_dense_matrix_amd")


@pytest.fixture(scope="module")
def S():
    import sparse_dense_matrix_amd as S
    return S


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    if not os.path.exists(os.path.join(LIBDIR, "libspmm.so")):
        pytest.skip("library not built")
    exe = str(tmp_path_factory.mktemp("attn") / "attn_driver")
    subprocess.run([hipcc, "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "attn_driver.cpp"), "-o", exe,
                    "-L", LIBDIR, "-lspmm", f"-Wl,-rpath,{LIBDIR}"], check=True, capture_output=True)

    def ask(*lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        return r.stdout.rstrip("\n").split("\n")
    return ask


def test_lengths_positions_and_pages_stay_inside(ask):
    big = 2 ** 31 - 1
    assert ask("len -5 100", "len 0 100", "len 100 100", f"len {big} 100", f"len {-big - 1} 100") == \
        ["0", "0", "100", "100", "0"]
    assert ask("start 0 8 100", "start -3 8 100", f"start {-big - 1} 8 100", f"start {big} 8 100") == \
        ["0", "-3", "-8", "100"]
    assert ask("page 1 4 3 0 3 2", "page 1 4 3 0 4 2", "page 1 4 3 0 -1 2", f"page 1 4 3 0 {big} 2",
               f"page 0 4 3 {-big - 1} 0 0", "page 7 4 0") == ["3", "-1", "-1", "-1", "-1", "7"]
    assert ask("names 0 0", "names 1 63", "names 1 64", "names -1 64", "names 0 -1", f"names {big} 1000",
               f"names {-big - 1} 1000") == ["1", "0", "1", "0", "0", "0", "0"]


def test_plan_cuts_lists_and_rows_completely(ask):
    r = np.random.default_rng(0)
    for _ in range(60):
        hk = int(r.choice([1, 2, 4, 8]))
        group = int(r.choice([1, 2, 3, 5, 8, 16, 100]))
        q_block = int(r.choice([1, 2, 4, 8, 16, 32, 64]))
        b, nq, nk = int(r.integers(1, 40)), int(r.integers(1, 5000)), int(r.integers(1, 40000))
        blocks = int(r.integers(1, 400))
        out = ask(f"plan {b} {nq} {nk} {hk * group} {hk} 128 {q_block} {blocks} 1")[0].split()
        assert out[0] == "SPMM_OK"
        rows, rtiles, tile, nsplit, per, chunk, slots = map(int, out[1:])
        assert rows == min(q_block, nq) * group and rtiles * tile >= rows > (rtiles - 1) * tile
        assert nsplit * per >= blocks and (nsplit - 1) * per < blocks
        assert 1 <= chunk <= 1024 and (chunk == 1 or chunk * rows <= 2 ** 28)
        # key blocks' items start at kb + (entries before) / chunk: none overlap, all fit
        nkb, entries = -(-nk // 64), -(-nq // q_block) * blocks
        assert slots == nkb + entries // chunk
        same = r.multinomial(int(r.integers(0, entries + 1)), r.dirichlet(np.full(nkb, 0.05)))
        less = np.concatenate([[0], np.cumsum(same)])
        first = np.arange(nkb) + less[:-1] // chunk
        end = first + np.maximum(1, -(-same // chunk))
        assert (end[:-1] <= first[1:]).all() and end[-1] <= slots


BAD_SHAPES = [
    (dict(batch=-1), "INVALID_ARG"), (dict(queries=2 ** 31), "INVALID_ARG"), (dict(keys=-1), "INVALID_ARG"),
    (dict(heads_q=3, heads_kv=2), "INVALID_ARG"), (dict(heads_kv=0), "INVALID_ARG"), (dict(q_block=0), "INVALID_ARG"),
    (dict(max_blocks=0), "INVALID_ARG"), (dict(local_blocks=0), "INVALID_ARG"), (dict(sink_blocks=-1), "INVALID_ARG"),
    (dict(scale=float("inf")), "INVALID_ARG"), (dict(dim=80), "UNSUPPORTED"), (dict(dim=256), "UNSUPPORTED"),
    (dict(q_block=48), "UNSUPPORTED"), (dict(q_block=128), "UNSUPPORTED"), (dict(dtype="F32"), "UNSUPPORTED"),
    (dict(heads_q=2 ** 17, heads_kv=1), "UNSUPPORTED"), (dict(batch=2 ** 20, queries=2 ** 20, q_block=1), "UNSUPPORTED"),
]


@pytest.mark.parametrize("change,status", BAD_SHAPES, ids=[str(c) for c, _ in BAD_SHAPES])
def test_plan_refuses(S, change, status):
    kw = dict(batch=1, queries=64, keys=64, heads_q=4, heads_kv=2, dim=64)
    kw.update(change)
    if "dtype" in kw:
        kw["dtype"] = getattr(S, kw["dtype"])
    with pytest.raises(S.SpmmError) as e:
        S.spmm_plan_attn(**kw)
    assert e.value.name == "SPMM_ERR_" + status and "spmm_plan_attn" in e.value.message


@pytest.mark.parametrize("scale", [-1.0, 0.0, float("nan")])
def test_binding_refuses_scales(S, scale):
    with pytest.raises(ValueError):
        S.spmm_plan_attn(1, 64, 64, 4, 2, 64, scale=scale)


REFUSED = {
    "q_null": "q is NULL", "q_null_tensor": "q is NULL", "q_odd": "16-byte", "q_stride_odd": "multiples of 8",
    "q_stride_negative": "multiples of 8", "q_stride_huge": "too large", "k_stride_short": "token stride",
    "k_stride_wide": "token stride", "o_overlaps": "must not overlap", "o_heads_overlap": "must not overlap",
    "lens_odd": "lens is not aligned", "lse_null": "lse is NULL", "lists_null": "lists is NULL",
    "pages_negative": "pages must be", "pages_huge": "pages must be", "tree_long": "at most 64",
    "tree_odd": "tree is not aligned", "select_short_list": "at most max_blocks", "select_long": "32768",
    "pool_odd": "pooled is not aligned", "no_plan": "plan is NULL", "other_plan": "not an attention plan",
    "execute": "", "no_backward": "without backward", "dq_null": "dq is NULL", "dk_broadcast": "must not overlap",
    "g_wide": "4 GiB",
}


def test_executes_refuse(ask):
    got = ask(*[f"refuse {c}" for c in REFUSED])
    for (c, text), line in zip(REFUSED.items(), got):
        status, _, message = line.partition(" ")
        want = "SPMM_ERR_UNSUPPORTED" if c in ("k_stride_short", "k_stride_wide", "tree_long", "select_long", "g_wide") \
            else "SPMM_ERR_INVALID_ARG"
        assert status == want and text in message, (c, line)
    assert ask("refuse nothing")[0].split()[0] == "SPMM_OK"  # no sequence: nothing to do, nothing touched


def test_reference_gradients_against_differences():
    """Central differences of sum(grad * o) in 64 bits: their error is of the
    order h^2 |f'''| + 2^-53 |f| / h, about 1e-9 of the gradients' size here."""
    c = dict(b=1, nq=24, nk=80, hq=4, hk=2, d=64, dtype=torch.float16, q_block=8, blocks=2)
    g = torch.Generator().manual_seed(1)
    q, k, v, grad = (torch.randn((1, n, h, 64), generator=g, dtype=torch.float64)
                     for n, h in ((24, 4), (80, 2), (80, 2), (24, 4)))
    lists = torch.tensor([[[[0, 1], [1, -1], [-1, -1]], [[0, -1], [0, 1], [1, -1]]]], dtype=torch.int32)
    w = R.sees(c, lists, [78], [60], None)
    want = R.attention(c, q, k, v, w, grad)

    def f(q, k, v):
        return (grad * R.attention(c, q, k, v, w)["o"][0]).sum().item()

    h = 1e-5
    for n, x in enumerate((q, k, v)):
        name = ("dq", "dk", "dv")[n]
        for _ in range(5):
            to = torch.randn(x.shape, generator=g, dtype=torch.float64)
            up, down = [q, k, v], [q, k, v]
            up[n], down[n] = x + h * to, x - h * to
            slope = (f(*up) - f(*down)) / (2 * h)
            want_slope = (want[name][0] * to).sum().item()
            size = (want[name][0].norm() * to.norm()).item()
            assert abs(slope - want_slope) <= 1e-7 * size, (name, slope, want_slope)


@pytest.mark.parametrize("blocks", [2 ** 30 + 1, 2 ** 31 - 1])
def test_plan_refuses_lists_that_kernels_cannot_count(S, blocks):
    """The kernels step through a list 64 or 256 entries at a time in 32 bits:
    from 2^31 - 256 entries on a step would wrap and never end."""
    with pytest.raises(S.SpmmError) as e:
        S.spmm_plan_attn(1, 64, 64, 4, 2, 64, max_blocks=blocks)
    assert e.value.name == "SPMM_ERR_UNSUPPORTED" and "max_blocks" in e.value.message


def test_plan_takes_long_lists(ask):
    assert ask(f"plan 1 64 640 4 2 64 64 {2 ** 30} 0")[0].split()[0] == "SPMM_OK"


@pytest.mark.parametrize("queries,keys", [(64, 2 ** 31 - 257), (2 ** 30, 2 ** 30)])
def test_plan_refuses_positions_past_32_bits(S, ask, queries, keys):
    """starts + t reaches queries + keys, and a row tile 256 more: the last key
    that a tile sees would wrap to a negative one, and its rows see nothing."""
    with pytest.raises(S.SpmmError) as e:
        S.spmm_plan_attn(1, queries, keys, 4, 2, 64)
    assert e.value.name == "SPMM_ERR_UNSUPPORTED" and "queries + keys" in e.value.message
    assert ask(f"plan 1 64 {2 ** 31 - 600} 4 2 64 64 16 0")[0].split()[0] == "SPMM_OK"


def test_written_tensors_must_not_overlap(ask):
    """Every small layout: refused where two rows share an element, and only there."""
    r = np.random.default_rng(3)
    lines, want = [], []
    layouts = [(1, 4, 4, 0, 64, 64), (2, 3, 4, 256, 64, 128), (1, 2, 3, 0, 192, 128), (3, 2, 2, 64, 192, 384),
               (2, 5, 1, 64, 128, 64), (4, 1, 1, 0, 64, 64), (1, 1, 1, 0, 0, 0), (2, 3, 4, 64, 512, 128)]
    layouts += [(*r.integers(1, 5, 3).tolist(), *(8 * r.integers(0, 80, 3)).tolist()) for _ in range(600)]
    layouts += [(*r.integers(1, 5, 3).tolist(), *(64 * r.integers(0, 20, 3)).tolist()) for _ in range(600)]
    for b, nq, hq, sb, st, sh in layouts:
        starts = np.sort((np.arange(b)[:, None, None] * sb + np.arange(nq)[:, None] * st + np.arange(hq) * sh).ravel())
        want.append("o is written" if (np.diff(starts) < 64).any() else "lse is NULL")
        lines.append(f"written {b} {nq} {hq} {sb} {st} {sh}")
    # large ones: nested in any order, interleaved, and heads on top of tokens
    for line, text in (("1000 100000 64 409600000 4096 64", "lse"), ("1000 100000 64 4096 4096000 64", "lse"),
                       ("64 4096 32 64 131072 4096", "lse"), ("1 100000 64 0 64 64", "o is written"),
                       ("2 100000 64 409599936 4096 64", "o is written")):
        lines.append("written " + line)
        want.append(text)
    got = ask(*lines)
    assert len(got) == len(want)
    bad = [(x, y, z) for x, y, z in zip(lines, want, got) if y not in z]
    assert not bad, bad[:5]
