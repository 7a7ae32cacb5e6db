"""The waits around the MFMAs that are written as inline assembly (csrc/tile_product.h):
the compiler neither sees that one writes its sums late nor keeps a VALU write of an
operand away from it.  So the built library is read back, kernel by kernel and along
every branch, and has to show that

* what an MFMA writes is touched by nothing but MFMAs that add to the very same sums
  for SETTLED wait states (more than an MFMA of 16 passes needs; these take fewer), and
* two wait states lie between a VALU write of a register and an MFMA that reads it.

An instruction counts as one wait state, s_nop n as n + 1.
"""
import os
import re
import shutil
import subprocess

import pytest

from bit_moe_decode_amd import build as build_mod

LLVM = "/opt/rocm/llvm/bin"
SETTLED, WRITTEN = 20, 2
# the kernels of the tiles whose MFMAs are inline assembly
KERNELS = ("moe_product_kernel", "moe_product_dw_kernel", "lm_loss_kernel", "lm_loss_d_kernel",
           "lm_loss_products_kernel")

REG = re.compile(r"\b([av])(?:\[(\d+):(\d+)\]|(\d+)\b)")
LINE = re.compile(r"^\s+(\S+)\s*(.*?)\s*//\s*([0-9A-F]+):(?:.*<\S+?(?:\+0x([0-9a-f]+))?>)?")


def registers(text):
    out = set()
    for kind, lo, hi, one in REG.findall(text):
        out.update((kind, i) for i in range(int(lo or one), int(hi or one) + 1))
    return out


class Instruction:
    def __init__(self, op, args, at, target):
        self.op, self.at, self.target = op, at, target
        args = args.split(",")
        self.mfma = op.startswith("v_mfma")
        self.all = registers(",".join(args))
        self.first = frozenset(registers(args[0]))
        self.a_b = registers(",".join(args[1:3])) if self.mfma else set()
        self.c = frozenset(registers(args[3])) if self.mfma else frozenset()
        swap = "swap" in op
        valu = op.startswith("v_") and not self.mfma
        self.written = (registers(",".join(args[:2])) if swap else self.first) if valu else ()
        self.states = int(args[0], 0) + 1 if op == "s_nop" else 1
        self.text = f"{at:x}: {op} {','.join(args)}"


def kernels(listing):
    """{name: instructions} of a disassembly."""
    out, start = {}, 0
    for line in listing.splitlines():
        head = re.match(r"^([0-9a-f]+) <(\S+)>:", line)
        if head:
            now, start = out.setdefault(head.group(2), []), int(head.group(1), 16)
            continue
        m = LINE.match(line)
        if m:
            op, args, at, off = m.groups()
            branch = op.startswith(("s_cbranch", "s_branch"))
            now.append(Instruction(op, "" if branch else args, int(at, 16),
                                   start + int(off or "0", 16) if branch else None))
    return out


def problems(code):
    """What breaks the two rules in a kernel, along every path through it."""
    index = {i.at: n for n, i in enumerate(code)}
    begins = {0} | {index[i.target] for i in code if i.target is not None}
    begins |= {n + 1 for n, i in enumerate(code[:-1]) if i.target is not None or i.op == "s_endpgm"}
    found = {}
    seen = {}  # block -> the youngest sums and VALU writes at its start
    todo = [(0, ({}, {}))]
    while todo:
        n, (sums, writes) = todo.pop()
        old = seen.get(n)
        if old is not None:
            merged = tuple({r: min(a.get(r, (99,)), b.get(r, (99,))) for r in {*a, *b}}
                           for a, b in zip(old, (sums, writes)))
            if merged == old:
                continue
            sums, writes = merged
        seen[n] = (dict(sums), dict(writes))
        sums, writes = dict(sums), dict(writes)
        while True:
            i = code[n]
            late = {r for r in i.all if r in sums}
            if i.mfma:
                mine = i.first if i.first == i.c else frozenset()
                if any(sums[r][1] != mine or r in i.a_b for r in late):
                    found[i.text] = "reads or writes sums under way"
                if any(r in writes for r in i.a_b | i.c):
                    found[i.text] = "an operand was written just before"
            elif late:
                found[i.text] = "touches sums under way"
            sums = {r: (age + i.states, of) for r, (age, of) in sums.items() if age + i.states < SETTLED}
            writes = {r: (age + i.states,) for r, (age,) in writes.items() if age + i.states < WRITTEN}
            if i.mfma:
                sums.update((r, (0, i.first)) for r in i.first)
            writes.update((r, (0,)) for r in i.written)
            if i.target is not None:
                todo.append((index[i.target], (sums, writes)))
            if i.op in ("s_endpgm", "s_branch"):
                break
            n += 1
            if n in begins:
                todo.append((n, (sums, writes)))
                break
    return found


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    """The kernels of the built library."""
    if not os.path.exists(build_mod.LIB):
        build_mod.build()
    where = tmp_path_factory.mktemp("code")
    copy = shutil.copy(build_mod.LIB, where / "lib.so")
    subprocess.run([f"{LLVM}/llvm-objdump", "--offloading", copy], check=True, capture_output=True, cwd=where)
    out = {}
    for f in sorted(where.glob(f"*{build_mod.ARCH}")):
        r = subprocess.run([f"{LLVM}/llvm-objdump", "-d", "--no-show-raw-insn", f], check=True, capture_output=True,
                           text=True)
        out.update({k: c for k, c in kernels(r.stdout).items() if any(re.search(rf"\d{n}", k) for n in KERNELS)})
    return out


def test_waits_around_the_tiles_mfmas(built):
    for name in KERNELS:
        assert any(name in k for k in built), name
    for k, code in built.items():
        assert sum(i.mfma for i in code) >= 16, k
        found = problems(code)
        assert not found, (k, list(found.items())[:5])


def _code(*lines):
    body = "".join(f"\t{t} // {4 * n:012X}: 00000000{' <k+0x%x>' % to if to is not None else ''}\n"
                   for n, (t, to) in enumerate(lines))
    return kernels(f"0000000000000000 <k>:\n{body}")["k"]


MFMA = ("v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]", None)
READ, WAIT, END = ("v_accvgpr_read_b32 v9, a2", None), ("s_nop 15", None), ("s_endpgm", None)


@pytest.mark.parametrize("lines,bad", [
    ([MFMA, MFMA, WAIT, WAIT, READ, END], 0),
    ([MFMA, WAIT, READ, END], 1),                                      # 17 states
    ([MFMA, ("buffer_store_dwordx4 a[0:3], v8, s[0:3], 0 offen", None), END], 1),
    ([MFMA, ("v_mfma_f32_16x16x32_bf16 a[2:5], v[0:3], v[4:7], a[2:5]", None), END], 1),
    ([MFMA, ("v_mfma_f32_16x16x32_bf16 a[8:11], a[0:3], v[4:7], a[8:11]", None), END], 1),
    ([("v_mov_b32_e32 v2, v8", None), MFMA, END], 1),
    ([("v_mov_b32_e32 v2, v8", None), WAIT, MFMA, END], 0),
    ([("v_permlane16_swap_b32_e32 v8, v5", None), MFMA, END], 1),
    ([("v_accvgpr_write_b32 a3, 0", None), ("s_nop 0", None), MFMA, END], 1),
    ([READ, MFMA, ("s_cbranch_scc1 65533", 0), WAIT, WAIT, READ, END], 1),  # along the branch back
    ([READ, MFMA, WAIT, WAIT, ("s_cbranch_scc1 65531", 0), END], 0),
    ([MFMA, ("s_cbranch_scc0 2", 16), WAIT, WAIT, READ, END], 1),      # past the wait
])
def test_what_the_reading_finds(lines, bad):
    assert len(problems(_code(*lines))) == bad
