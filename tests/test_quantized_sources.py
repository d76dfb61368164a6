"""What the assembly of the 8-bit integer kernels tells the compiler that it overwrites."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_ep_layout_amd", "csrc")


def test_assembly_that_writes_m0_says_so():
    found = 0
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for statement in re.findall(r"\basm volatile\((.*?)\);", text, re.S):
            if re.search(r"s_mov_b32 m0\b", statement):
                found += 1
                assert '"m0"' in statement.rsplit(":", 1)[1], f"{name}: {statement}"
    assert found
