"""Wait states that inline asm has to bring itself, checked in the compiled
kernels (CPU only; the disassembly of the library built here).

The compiler inserts the wait states that the hardware asks for between its
own instructions, but not inside an inline asm string, and not in front of one
for the registers it reads.  The direct loads to LDS are such strings.  They
need one wait state between a write of M0 and the load that takes its LDS
address from there, and five between a vector instruction that writes a scalar
register (v_readfirstlane and the like) and the load that reads it."""
import collections
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sparse_dense_matrix_amd", "libspmm.so")
OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"

INSN = re.compile(r"^\t(\S+)\s*(.*?)\s*// ([0-9A-F]+):")
FUNC = re.compile(r"^([0-9a-f]+) <(.+)>:")
TARGET = re.compile(r"<[^<>]+?(?:\+0x([0-9a-f]+))?>\s*$")

Insn = collections.namedtuple("Insn", "op args target")


def functions(listing):
    """{name: [Insn]} of a disassembly; a target is an index into the list."""
    out = {}
    base = rows = None
    for line in listing.splitlines():
        m = FUNC.match(line)
        if m:
            base, rows = int(m[1], 16), out.setdefault(m[2], [])
            continue
        m = INSN.match(line)
        if m and rows is not None:
            t = TARGET.search(line) if m[1].startswith(("s_branch", "s_cbranch")) else None
            rows.append((int(m[3], 16), m[1], m[2], base + int(t[1] or "0", 16) if t else None))
    for name, rows in out.items():
        at = {a: i for i, (a, *_) in enumerate(rows)}
        out[name] = [Insn(op, args, None if t is None else at[t]) for _, op, args, t in rows]
    return out


def scalars(text):
    """Scalar registers that operands name."""
    out = set()
    for m in re.finditer(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        out |= set(range(int(m[1] or m[3]), int(m[2] or m[3]) + 1))
    return out | {r for r in ("m0", "vcc") if re.search(rf"\b{r}\b", text)}


def written(insn):
    """Scalar registers that an instruction writes."""
    ops = insn.args.split(", ")
    if insn.op.startswith("v_"):
        out = scalars(ops[0])
        if re.match(r"v_(add_co|sub_co|subrev_co|addc|subb|subbrev|div_scale|mad_[ui]64)", insn.op) and len(ops) > 1:
            out |= scalars(ops[1])
        return out
    if insn.op.startswith("s_") and not re.match(r"s_(cmp|bitcmp|cbranch|branch|waitcnt|nop|barrier|endpgm|set|sleep)", insn.op):
        return scalars(ops[0])
    return set()


def is_lds_load(insn):
    return insn.op.startswith(("global_load_lds", "buffer_load_lds")) or \
        (insn.op.startswith("buffer_load") and re.search(r"\blds\b", insn.args) is not None)


def too_close(insns, i, regs, by, need):
    """Whether some path reaches insns[i] with a register of regs last written
    by an instruction that by() picks, fewer than `need` wait states before."""
    preds = collections.defaultdict(list)
    for j, x in enumerate(insns):
        if x.target is not None:
            preds[x.target].append(j)
        if x.op not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            preds[j + 1].append(j)
    work, seen = [(i, 0, frozenset(regs))], set()
    while work:
        at, states, regs = work.pop()
        for j in preds[at]:
            x = insns[j]
            hit = written(x) & regs
            if hit and by(x):
                return True
            left = regs - hit  # another write hides those before it
            n = states + (int(x.args.split()[0], 0) + 1 if x.op == "s_nop" else 1)
            if left and n < need and (j, n, left) not in seen:
                seen.add((j, n, left))
                work.append((j, n, left))
    return False


def m0_faults(insns):
    return [i for i, x in enumerate(insns) if is_lds_load(x) and too_close(insns, i, {"m0"}, lambda w: True, 1)]


def is_memory(insn):
    return insn.op.startswith(("global_", "buffer_", "flat_", "scratch_"))


def scalar_faults(insns):
    return [i for i, x in enumerate(insns)
            if is_memory(x) and too_close(insns, i, scalars(x.args), lambda w: w.op.startswith("v_"), 5)]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """[(name, instructions)] of every device function of the library."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump not found")
    if not os.path.exists(LIB):
        pytest.skip("library not built")
    d = tmp_path_factory.mktemp("isa")
    subprocess.run([OBJDUMP, "--offloading", shutil.copy(LIB, d)], cwd=d, check=True, capture_output=True)
    out = []
    for f in sorted(os.listdir(d)):
        if "gfx950" in f:
            r = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", os.path.join(d, f)], capture_output=True, text=True, check=True)
            out += functions(r.stdout).items()
    return out


LISTING = """
0000000000001000 <k>:
\ts_mov_b32 m0, s4                                           // 000000001000: BEFC0004
%s\tbuffer_load_dwordx4 v2, s[28:31], 0 offen lds              // 000000001008: E05D1000 80070002
\ts_cbranch_scc1 65533                                       // 000000001010: BF85FFFD <k+0x8>
\ts_endpgm                                                   // 000000001014: BF810000
"""


def test_the_check_itself():
    nop = "\ts_nop 0                                                    // 000000001004: BF800000\n"
    assert m0_faults(functions(LISTING % "")["k"]) == [1]
    good = functions(LISTING % nop)["k"]
    assert m0_faults(good) == [] and good[3].target == 2


READ = """
0000000000001000 <k>:
\tv_readfirstlane_b32 s30, v7                                // 000000001000: 7E3C0507
%s\tv_lshl_add_u32 v2, v3, 4, v2                               // 000000001010: D1FD0002 04090903
\ts_mov_b32 m0, s4                                           // 000000001018: BEFC0004
\tbuffer_load_dwordx4 v2, s[28:31], 0 offen lds              // 00000000101C: E05D1000 80070002
\ts_endpgm                                                   // 000000001024: BF810000
"""


def test_the_check_of_scalar_operands():
    for between, faults in (("", [3]), ("\ts_nop 1    // 000000001004: BF800001\n", [4]),
                            ("\ts_nop 2    // 000000001004: BF800002\n", []),
                            ("\ts_mov_b32 s30, 0    // 000000001004: BE9E0080\n", [])):
        assert scalar_faults(functions(READ % between)["k"]) == faults, between


def test_loads_wait_for_scalars_from_vector_instructions(kernels):
    bad = {name: len(f) for name, insns in kernels if (f := scalar_faults(insns))}
    assert not bad, bad


def test_lds_loads_wait_for_m0(kernels):
    loads = [(name, sum(is_lds_load(x) for x in insns)) for name, insns in kernels]
    assert sum(n for _, n in loads) > 500, "the library's direct loads were not found"
    bad = {name: len(f) for name, insns in kernels if (f := m0_faults(insns))}
    assert not bad, bad
