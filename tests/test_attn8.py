"""What stands around attention over a cache, on the CPU: the refusals of every
call (tests/attn8_driver.cpp drives the library without a device), the
binding's checks, and the reference that the GPU tests use."""
import os
import shutil
import struct
import subprocess
import sys

import numpy as np
import pytest
import torch

import attn8_ref as R

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
    exe = str(tmp_path_factory.mktemp("attn8") / "attn8_driver")
    subprocess.run([hipcc, "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "attn8_driver.cpp"), "-o", exe,
                    "-L", LIBDIR, "-lspmm", f"-Wl,-rpath,{LIBDIR}"], check=True, capture_output=True)

    def ask(*lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        return r.stdout.rstrip("\n").split("\n")
    return ask


SHARED = {"no_plan": "plan is NULL", "other_plan": "not an attention plan", "k8_null": "k8 is NULL",
          "k8_odd": "16-byte", "k8_stride_odd": "multiples of 16", "k8_stride_wide": "token stride",
          "ks_null": "k_scale is NULL", "ks_odd": "k_scale is not aligned", "lens_odd": "lens is not aligned",
          "pages_negative": "pages must be", "table_odd": "table is not aligned"}
OWN = {"write": {"k_null": "k is NULL", "k8_overlaps": "must not overlap", "v8_null": "v8 is NULL",
                 "vs_null": "v_scale is NULL", "starts_odd": "starts is not aligned", "many_rows": "more workgroups"},
       "read": {"k_null": "k is NULL", "k_overlaps": "must not overlap", "v8_null": "v8 is NULL",
                "vs_null": "v_scale is NULL", "many_rows": "more workgroups"},
       "pool8": {"pooled_odd": "pooled is not aligned", "vs_null": "pooled_scale is NULL",
                 "starts_odd": "first is not aligned"},
       "cache8": {"v8_null": "v8 is NULL", "vs_null": "v_scale is NULL", "starts_odd": "starts is not aligned",
                  "tree_long": "at most 64"}}


@pytest.mark.parametrize("call", OWN)
def test_cache_calls_refuse(ask, call):
    cases = {**SHARED, **OWN[call]}
    for (what, text), line in zip(cases.items(), ask(*[f"{call} {what}" for what in cases])):
        status, _, message = line.partition(" ")
        want = "SPMM_ERR_UNSUPPORTED" if what in ("k8_stride_wide", "many_rows", "tree_long") else "SPMM_ERR_INVALID_ARG"
        assert status == want and text in message and f"spmm_execute_attn_{call}" in message, (what, line)
    assert ask(f"{call} nothing")[0].split()[0] == "SPMM_OK"  # no sequence: nothing to do, nothing touched


ROPE = {"batch": "batch", "tokens": "tokens", "too_many": "batch * tokens", "heads": "heads", "heads_many": "heads",
        "pairs": "pairs must be 0", "pairs_odd": "multiple of 8", "axes": "axes", "axis": "axis must be", "eps": "eps",
        "eps_nan": "eps", "freqs_null": "freqs is NULL", "freqs_nan": "finite", "dim": "64 or 128", "dtype": "bf16 or f16",
        "interleaved": "interleaved", "no_plan": "plan is NULL", "other_plan": "not a rotation plan",
        "execute": "rotation plan", "sddmm": "not an SDDMM plan", "attn": "not an attention plan", "q_null": "q is NULL",
        "q_stride": "multiples of 8", "k_odd": "16-byte", "out_null": "is NULL", "out_overlaps": "must not overlap",
        "weight_odd": "q_weight is not aligned", "positions_odd": "positions is not aligned", "lens_odd": "lens is not aligned"}
BACK = {"no_backward": "without backward", "dw_null": "dk_weight is NULL", "dw_without": "weight that is NULL",
        "grad_null": "q_grad is NULL"}
UNSUPPORTED = ("too_many", "heads_many", "pairs_odd", "dim", "dtype")


@pytest.mark.parametrize("call", ["rope", "rope_backward"])
def test_rope_calls_refuse(ask, call):
    cases = {**ROPE, **(BACK if call == "rope_backward" else {})}
    for (what, text), line in zip(cases.items(), ask(*[f"{call} {what}" for what in cases])):
        status, _, message = line.partition(" ")
        want = "SPMM_ERR_UNSUPPORTED" if what in UNSUPPORTED else "SPMM_ERR_INVALID_ARG"
        assert status == want and text in message, (what, line)
    assert ask("rope nothing")[0].split()[0] == "SPMM_OK"


def test_writing_and_reading_back_hold_what_a_launch_does(ask):
    """2^24 workgroups or more are refused before any of them starts."""
    for what in ("write rows_launch", "write blocks_launch", "read blocks_launch"):
        status, _, message = ask(what)[0].partition(" ")
        assert status == "SPMM_ERR_UNSUPPORTED" and "more workgroups than a launch holds" in message, (what, message)


def test_rope_plans_hold_what_a_launch_does(ask):
    """2^24 - 1 workgroups of 256 threads, of 4 tokens (more than 16 heads) or 16:
    one row of tokens more is refused before the first call."""
    for what, limit in (("launch", 4 * (2 ** 24 - 1)), ("launch_few", 16 * (2 ** 24 - 1))):
        status, _, message = ask(f"rope {what}")[0].partition(" ")
        assert status == "SPMM_ERR_UNSUPPORTED" and str(limit) in message, message
        assert ask(f"rope {what}_holds")[0].split()[0] == "SPMM_OK"


def test_binding_refuses(S):
    with pytest.raises(ValueError):
        S.spmm_plan_attn_rope(1, 4, 2, 1, 64, [[1.0] * 8])
    with pytest.raises(ValueError):
        S.spmm_plan_attn_rope(1, 4, 2, 1, 64, [1.0] * 8, axis=[0] * 7)
    with pytest.raises(S.SpmmError) as e:
        S.spmm_plan_attn_rope(1, 4, 2, 1, 64, [1.0] * 8, axis=[0] * 7 + [2], axes=2)
    assert e.value.name == "SPMM_ERR_INVALID_ARG" and "axis" in e.value.message


def test_tensor_checks_without_the_module(S, monkeypatch):
    """Without csrc/binding.cpp's module (a library given alone), or with one of
    another torch, the checks run in Python: what fits goes on, the rest is refused."""
    if not os.path.exists(os.path.join(LIBDIR, "_binding.so")):
        pytest.skip("module not built")
    monkeypatch.setattr(S, "_bind", None)
    module = S._load_binding()
    assert module.__name__.endswith("_binding") and module.torch_version == torch.__version__.split("+")[0]
    monkeypatch.setattr(module, "torch_version", "1.0.0")
    assert S._load_binding() is S._PythonChecks
    monkeypatch.delattr(S, "_binding")
    monkeypatch.setitem(sys.modules, S.__name__ + "._binding", None)
    monkeypatch.setattr(S, "_bind", None)
    x = torch.zeros((2, 3, 8, 64), dtype=torch.bfloat16)
    want, here = ((2, 3, 4, 64), torch.bfloat16), -1  # the device of CPU tensors
    y = x[:, :, 4:]
    assert struct.unpack("=4q", S._heads("q", y, want, here)) == (y.data_ptr(), 3 * 512, 512, 64)
    assert S._bind is S._PythonChecks
    for bad in (x, y.half(), y.transpose(2, 3).contiguous().transpose(2, 3)):
        with pytest.raises(ValueError):
            S._heads("q", bad, want, here)
    with pytest.raises(ValueError):
        S._heads("q", y, want, 0)
    assert S._flat("k", y.contiguous(), want, here) and S._opt("k", None, want, here) is None
    for bad in (y, y.contiguous().half(), x):
        with pytest.raises(ValueError):
            S._flat("k", bad, want, here)


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_gradients_against_differences(interleaved):
    """Central differences of sum(grad * o) in 64 bits: their error is of the
    order h^2 |f'''| + 2^-53 |f| / h, about 1e-9 of the gradients' size here."""
    g = torch.Generator().manual_seed(5)
    x, grad = (torch.randn((2, 3, 4, 64), generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.randn(64, generator=g, dtype=torch.float64)
    place = torch.randint(-50, 5000, (2, 2, 3), generator=g)
    a, off = R.angles(R.freqs(24), [p % 2 for p in range(24)], place)
    alive = torch.tensor([[1, 1, 0], [1, 1, 1]], dtype=torch.bool)
    kw = dict(angle=a, off=off, interleaved=interleaved, eps=1e-6, dtype=torch.bfloat16)
    want = R.rope(x, w, grad=grad, alive=alive, **kw)

    def f(x, w):
        return (torch.where(alive[..., None, None], grad, 0.0) * R.rope(x, w, **kw)["o"][0]).sum().item()

    h = 1e-5
    for _ in range(5):
        to, tow = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(64, generator=g, dtype=torch.float64)
        slope = (f(x + h * to, w) - f(x - h * to, w)) / (2 * h)
        assert abs(slope - (want["dx"][0] * to).sum().item()) <= 1e-7 * (want["dx"][0].norm() * to.norm()).item()
        slope = (f(x, w + h * tow) - f(x, w - h * tow)) / (2 * h)
        assert abs(slope - (want["dw"][0] * tow).sum().item()) <= 1e-7 * (want["dw"][0].norm() * tow.norm()).item()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_codes_survive_a_32_bit_division(dtype):
    """The kernel rounds a correctly rounded 32-bit quotient; the reference the
    number itself, in whole numbers: equal for every pair of significands, at
    every distance of the exponents that leaves a code."""
    bits = 8 if dtype == torch.bfloat16 else 11
    tops = np.arange(2 ** (bits - 1), 2 ** bits, dtype=np.int64)
    for shift in range(8):
        for top in tops[::1 if bits == 8 else 7]:
            x = np.arange(2 ** bits, dtype=np.int64)
            x = x[x <= top << shift]
            n, m = 254 * x + (top << shift), 2 * (top << shift)
            want = n // m - ((n % m == 0) & (n // m % 2 == 1))  # half up, and ties to even
            got = np.rint(np.float32(127) * x.astype(np.float32) / np.float32(top << shift))
            assert (got == want).all()


def test_tokens_go_to_their_blocks(tmp_path):
    """Each position in [0, len) once, in its block, and nothing else: at every
    32-bit start (idle sequences are often marked by one of its ends)."""
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not found")
    exe = str(tmp_path / "taken")
    subprocess.run([hipcc, "-O1", "-std=c++17", os.path.join(ROOT, "tests", "attn_taken_driver.cpp"), "-o", exe],
                   check=True, capture_output=True)
    least, most = -2 ** 31, 2 ** 31 - 1
    rng = np.random.default_rng(7)
    starts = [least + d for d in (0, 1, 60, 61, 62, 63, 64, 1000)] + [most - d for d in (0, 1, 62, 63, 64, 129, 4096)]
    starts += [-1000, -65, -64, -1, 0, 1, 63, 64, 65, 4000] + rng.integers(-3000, 6000, 40).tolist()
    cases = [(s, n, n_i) for s in starts for n in (65, 66, 127, 1000, 4097) for n_i in (0, 1, 10, 64, 777, 4096, most - 256)]
    rows, lines = [], []
    for s, n, n_i in cases:
        width = (n + 62) // 64 + 1
        rows += [(s, n, n_i)] * width
        lines += [f"{s} {n} {n_i} {w}" for w in range(width)]
    out = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True).stdout.split("\n")
    taken = {c: [] for c in cases}
    for c, line in zip(rows, out):
        block, lo, hi = map(int, line.split())
        assert lo >= hi or (0 <= lo and hi <= 64 and block >= 0), (c, line)
        taken[c] += range(block * 64 + lo, block * 64 + hi)
    for (s, n, n_i), got in taken.items():
        assert got == list(range(max(s, 0), min(s + n, n_i))), (s, n, n_i)


def test_reference_codes():
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5, 0.25, -127.0], [0.0] * 6, [1.0, float("nan"), 0, 0, 0, 0]])
    code, scale = R.encode(x.to(torch.bfloat16))
    assert code.tolist() == [[127, 0, 2, -2, 0, -127], [0] * 6, [0] * 6]
    assert scale[0] == 1 and scale[1] == 0 and scale[2].isnan()
