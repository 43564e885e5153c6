"""Loads of tensor memory, from the source: their registers hold nothing before the wait, which names none of them.  So either
load and wait are one piece of assembly, or all that reads the registers is volatile, which keeps its place behind the wait."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_ep_layout_03_gb300", "csrc")


def sources():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            yield os.path.basename(path), re.sub(r"//.*", "", f.read())


def test_loads_that_wait_are_one_piece():
    text = dict(sources())["tcgen05.cuh"]
    body = text[text.index("void tmem_load32("):]
    body = body[:body.index("\n}\n")]
    assert body.count("asm volatile") == 1 and "tcgen05.ld." in body and "tcgen05.wait::ld" in body
    # the only other load is the one whose readers are volatile
    assert sum(t.count('"tcgen05.ld.') for _, t in sources()) == 2


def test_readers_of_the_other_load_are_volatile():
    text = dict(sources())["matmul_fp8.cu"]
    assert all("tmem_start16" not in t for name, t in sources() if name not in ("matmul_fp8.cu", "tcgen05.cuh"))
    uses = re.findall(r"tmem_start16\(([^;]*), v\);(.*?)\n\s*}\n", text, re.S)
    assert len(uses) == 1
    readers = re.findall(r"(\w+)\([^;]*\bv\[i\]", uses[0][1])
    assert readers == ["add_scaled"]
    add = text[text.index("void add_scaled("):]
    assert "asm volatile" in add[:add.index("\n}\n")]
