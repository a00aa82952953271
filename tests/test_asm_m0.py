"""The copies from memory into LDS take their LDS address from m0, which their inline
assembly sets. It cannot be declared as overwritten: the compiler keeps the register
for itself and warns of such a declaration. So this test reads the gfx950 code of the
built library (disassembled with ROCm's llvm-objdump) and checks that nothing but those
statements names m0, and that each sets it right before its copy. CPU only."""
import re

from test_asm_scc import _disassemble


def test_only_the_copies_use_m0(tmp_path):
    lines = [l for l in _disassemble(tmp_path) if l]
    named = [i for i, l in enumerate(lines) if re.search(r"\bm0\b", l)]
    assert len(named) > 1000
    bad = [lines[i:i + 3] for i in named
           if not (re.match(r"s_(add_u32|mov_b32) m0, ", lines[i]) and lines[i + 1] == "s_nop 0"
                   and lines[i + 2].startswith("global_load_lds_"))]
    assert not bad, f"{len(bad)} other uses of m0, e.g. {bad[:2]}"
