"""Waits of the products' kernels that poll inside one piece of assembly: each poll is bounded in time, and so are all of
them together, by the clock and the limit that mbar_wait_parked() has (a count of polls of unknown length bounds nothing)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_ep_layout_03_gb300", "csrc")


def pieces():
    """(file, text) of each piece of assembly that waits and branches back."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            for block in re.findall(r"asm volatile\((.*?)\);\n", f.read(), re.S):
                if "mbarrier.try_wait" in block and re.search(r"\bbra\b", block):
                    yield os.path.basename(path), block


def test_polls_in_assembly_end_by_the_clock():
    found = list(pieces())
    assert any(name == "matmul_fp8.cu" for name, _ in found)
    for name, block in found:
        assert re.search(r"try_wait\.parity\.shared::cta\.b64 p, \[%\d\], %\d, %\d;", block), (name, "a poll without a time")
        assert "%%globaltimer" in block and '"l"(kWaitNs)' in block, (name, "polls without a clock")


def test_all_waits_of_the_products_have_one_limit():
    with open(os.path.join(CSRC, "tcgen05.cuh")) as f:
        text = f.read()
    assert "constexpr uint64_t kWaitNs = 4000000000ull;" in text and "now - start > kWaitNs" in text
