"""What inline assembly writes it names: a register that it sets without saying so
could be one that the compiler keeps something in."""
import os
import re

from memory_bound_gemv_row_amd import build


def test_written_scalar_registers_are_named():
    found = 0
    for name in sorted(os.listdir(build.SRC_DIR)):
        with open(os.path.join(build.SRC_DIR, name)) as f:
            text = f.read()
        for statement in re.findall(r"\basm\b.*?\);", text, re.S):
            for register in re.findall(r"s_mov_b32 (m0|vcc_lo|vcc_hi|exec_lo|exec_hi|s\d+)\b", statement):
                found += 1
                assert f'"{register}"' in statement, (name, statement)
    assert found    # the loads to LDS set m0
