"""Properties of the feed-forward kernels' sources that no call can show (no GPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "quantum_state_encoding_amd", "csrc")


def asm_statements(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.findall(r"\basm\s+volatile\s*\((.*?)\);", text, flags=re.S)


def test_asm_that_writes_m0_says_so():
    # the compiler may keep a value of its own in m0 across a statement that
    # does not name it
    found = 0
    for name in sorted(os.listdir(CSRC)):
        for body in asm_statements(name):
            if re.search(r"\bs_mov_b32 m0\b", body):
                found += 1
                clobbers = body.rsplit(":", 1)[1]
                assert '"m0"' in clobbers, (name, body)
    assert found >= 2
