"""The built library keeps the distances that its inline assembly needs (no GPU
needed); the reader itself on small listings with planted mistakes."""
import glob
import os
import re

import pytest

import built_code

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "combine_moe_dispatch_amd", "libmoe_dispatch.so")


@pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe_dispatch.so not built")
@pytest.mark.skipif(not os.path.exists(built_code.OBJDUMP), reason="no llvm-objdump")
def test_built_library(tmp_path):
    products = loads = 0
    for listing in built_code.disassemble(LIB, str(tmp_path)):
        wrong, p, n = built_code.check(listing)
        assert not wrong, wrong[:5]
        products, loads = products + p, loads + n
    assert products > 1000 and loads > 1000   # the listing was read


def listing(*lines):
    """lines: text, or (text, index of the line it branches to)."""
    out = ["0000000000001000 <kernel>:"]
    for i, line in enumerate(lines):
        text, to = line if isinstance(line, tuple) else (line, None)
        where = "" if to is None else f" <kernel+0x{4 * to:x}>" if to else " <kernel>"
        out.append(f"\t{text}   // {0x1000 + 4 * i:012X}: BF800000{where}")
    return "\n".join(out)


MFMA = "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]"
LOAD = "global_load_lds_dwordx4 v9, s[4:5]"


@pytest.mark.parametrize("wrong,lines", [
    (None, ["v_mov_b32_e32 v5, 0", "s_nop 1", MFMA, "s_endpgm"]),
    ("operand", ["v_mov_b32_e32 v5, 0", "s_nop 0", MFMA, "s_endpgm"]),
    ("operand", ["v_accvgpr_write_b32 a2, 0", MFMA, "s_endpgm"]),
    (None, ["v_mov_b32_e32 v8, v5", MFMA, "s_endpgm"]),
    (None, ["ds_read_b128 v[4:7], v8", MFMA, "s_endpgm"]),      # waited for by its counter
    ("operand", [MFMA, "v_mov_b32_e32 v0, 0", ("s_cbranch_scc1 0", 0), "s_endpgm"]),
    (None, [MFMA, "s_nop 7", "v_accvgpr_read_b32 v1, a1", "s_endpgm"]),
    ("result", [MFMA, "s_nop 6", "v_accvgpr_read_b32 v1, a1", "s_endpgm"]),
    ("result", [MFMA, ("s_cbranch_scc1 0", 3), "s_endpgm", "v_accvgpr_read_b32 v1, a1",
                "s_endpgm"]),
    (None, [MFMA, MFMA, "s_nop 7", "s_endpgm"]),
    (None, ["v_readfirstlane_b32 s4, v0", "s_mov_b32 m0, s6", "s_nop 3", LOAD, "s_endpgm"]),
    ("address", ["v_readfirstlane_b32 s4, v0", "s_mov_b32 m0, s6", "s_nop 2", LOAD, "s_endpgm"]),
    (None, ["v_readfirstlane_b32 s8, v0", "s_mov_b32 m0, s8", "s_nop 0", LOAD, "s_endpgm"]),
    ("m0", ["s_mov_b32 m0, s6", LOAD, "s_endpgm"]),
    ("packed", ["v_pk_fma_f32 v[0:1], v[2:3], v[4:5], v[6:7]", "s_endpgm"]),
])
def test_the_reader(wrong, lines):
    found, _, _ = built_code.check(listing(*lines))
    if wrong is None:
        assert not found
    else:
        assert len(found) == 1 and wrong in found[0]


def test_inline_assembly_names_the_registers_it_writes():
    """m0 is no output of a statement, so it has to be among its clobbers."""
    for path in glob.glob(os.path.join(ROOT, "combine_moe_dispatch_amd", "csrc", "*")):
        for asm in re.findall(r"asm volatile\((.*?)\);", open(path).read(), re.S):
            if re.search(r"\bm0\b", asm.split(":")[0]):
                assert '"m0"' in asm.rsplit(":", 1)[1], (path, asm)
