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
    # the only other loads are those whose readers are volatile
    assert sum(t.count('"tcgen05.ld.') for _, t in sources()) == 1 + len(re.findall(r"void tmem_start\d+\(", text))


def test_readers_of_the_other_loads_are_volatile():
    """Behind each such load, up to the end of its block: the wait, then nothing but assembly or add_scaled() reads v."""
    found = 0
    for name, text in sources():
        for use in re.finditer(r"tmem_start\d+\([^;{]*, v\);(.*?)\n\s*}\n", text, re.S):
            found += 1
            head, *readers = [x for x in re.sub(r'"[^"]*"', "", use.group(1)).split(";") if x.strip()]
            assert head.strip() == "tmem_wait_loads()", name
            for x in readers:
                assert not re.search(r"\bv\[", x) or "asm volatile(" in x or "add_scaled(" in x, (name, x)
    assert found == 2
    fp8 = dict(sources())["matmul_fp8.cu"]
    add = fp8[fp8.index("void add_scaled("):]
    assert "asm volatile" in add[:add.index("\n}\n")]
