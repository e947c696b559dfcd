"""Reads the disassembly of the built library and checks the distances that the
hardware wants around instructions written as inline assembly, which the
compiler's own hazard handling does not see.

Distances are wait states: every instruction is one, s_nop N is N + 1.  They are
followed over branches in both directions.
"""
import os
import re
import shutil
import subprocess

OBJDUMP = os.environ.get("LLVM_OBJDUMP", "/opt/rocm/llvm/bin/llvm-objdump")

VALU_TO_MATRIX = 2      # vector write -> operand of a matrix instruction
MATRIX_TO_USE = 8       # result of a 16 x 16 x 32 product (4 passes) -> anything but a product
VALU_SGPR_TO_LOAD = 5   # scalar register written by a vector instruction -> memory address
M0_TO_LOAD = 1          # m0 -> load to LDS

_REG = re.compile(r"\b([vas])\[(\d+):(\d+)\]|\b([vas])(\d+)\b|\b(m0)\b")


def registers(text):
    out = set()
    for m in _REG.finditer(text):
        if m.group(1):
            out |= {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
        elif m.group(4):
            out.add((m.group(4), int(m.group(5))))
        else:
            out.add((m.group(6), 0))
    return out


def disassemble(library, folder):
    """Listings of the library's device code objects."""
    copy = shutil.copy(library, os.path.join(folder, "library.so"))
    subprocess.run([OBJDUMP, "--offloading", copy], check=True, capture_output=True)
    for name in sorted(os.listdir(folder)):
        if "amdgcn" in name:
            r = subprocess.run([OBJDUMP, "-d", os.path.join(folder, name)], check=True,
                               capture_output=True, text=True)
            yield r.stdout


class Function:
    """Instructions of one function and which can follow which."""

    def __init__(self, name):
        self.name = name
        self.code = []   # (address, opcode, operands, offset of the branch target)

    def link(self):
        at = {c[0]: i for i, c in enumerate(self.code)}
        self.after = [[] for _ in self.code]
        self.before = [[] for _ in self.code]
        self.regs = [None] * len(self.code)
        for i, (_, op, _, target) in enumerate(self.code):
            follow = []
            if op.startswith("s_cbranch") or op == "s_branch":
                follow.append(at[self.code[0][0] + int(target or "0", 16)])
            if op not in ("s_branch", "s_endpgm") and i + 1 < len(self.code):
                follow.append(i + 1)
            for j in follow:
                self.after[i].append(j)
                self.before[j].append(i)

    def operands(self, i):
        if self.regs[i] is None:
            self.regs[i] = [registers(t) for t in self.code[i][2].split(",")]
        return self.regs[i]

    def near(self, i, edges, states, hit):
        """The first instruction within `states` of i along edges that hit names."""
        best, stack = {}, [(j, 0) for j in edges[i]]
        while stack:
            j, d = stack.pop()
            if d >= states or best.get(j, states) <= d:
                continue
            best[j] = d
            if hit(j):
                return j
            op, args = self.code[j][1:3]
            d += int(args, 0) + 1 if op == "s_nop" else 1
            stack += [(n, d) for n in edges[j]]
        return None


def functions(listing):
    out = []
    for line in listing.splitlines():
        m = re.match(r"^[0-9a-f]+ <(.+)>:$", line)
        if m:
            out.append(Function(m.group(1)))
            continue
        m = re.match(r"^\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+): [0-9A-F ]+(?:<\S+?(?:\+0x([0-9a-f]+))?>)?$",
                     line)
        if m and out:
            out[-1].code.append((int(m.group(3), 16), m.group(1), m.group(2), m.group(4)))
    for f in out:
        f.link()
    return out


def check(listing):
    """(what is wrong, matrix instructions, loads to LDS) of a listing."""
    wrong, products, loads = [], 0, 0
    for f in functions(listing):
        def name(i):
            return f"{f.code[i][0]:x}: {f.code[i][1]} {f.code[i][2]}"

        def report(what, i, j):
            if j is not None:
                wrong.append(f"{f.name}: {what}: {name(j)} / {name(i)}")

        def vector(j):
            return f.code[j][1].startswith("v_") and not f.code[j][1].startswith("v_mfma")

        def written_scalars(j):
            op = f.code[j][1]
            if op.startswith(("v_readlane", "v_readfirstlane", "v_cmp")):
                return f.operands(j)[0]
            if op.startswith("v_") and ("_co_" in op or "div_scale" in op):
                return f.operands(j)[1]
            return set()

        for i, (_, op, args, _) in enumerate(f.code):
            if op.startswith("v_mfma"):
                products += 1
                result, *sources = f.operands(i)
                sources = set().union(*sources)
                report("operand written too late", i,
                       f.near(i, f.before, VALU_TO_MATRIX,
                              lambda j: vector(j) and f.operands(j)[0] & sources))
                if "16x16x32" in op:
                    report("result used too early", i,
                           f.near(i, f.after, MATRIX_TO_USE,
                                  lambda j: not f.code[j][1].startswith(("v_mfma", "s_")) and
                                  set().union(*f.operands(j)) & result))
            elif op.startswith("global_load_lds"):
                loads += 1
                scalars = {r for r in registers(args) if r[0] == "s"}
                report("address written too late", i,
                       f.near(i, f.before, VALU_SGPR_TO_LOAD,
                              lambda j: written_scalars(j) & scalars))
                report("m0 written too late", i,
                       f.near(i, f.before, M0_TO_LOAD,
                              lambda j: ("m0", 0) in f.operands(j)[0]))
            elif re.match(r"v_pk_(add|mul|fma)_f32", op):
                wrong.append(f"{f.name}: packed fp32: {name(i)}")
    return wrong, products, loads
