"""The rows that are cleared behind a segment's end, on the CPU, from the source: they are ordinary writes of both CTAs of a
pair, and a thread of the first issues the products that read them.  The second CTA's word for it is a copy whose
completion is a release to the cluster, behind the fence between its writes and asynchronous reads; a plain arrival is
one of its own CTA only."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_ep_layout_03_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"\s+", " ", re.sub(r"//.*", "", f.read()))


def function(name, file="matmul_bf16.cu"):
    text = source(file)
    start = text.index(f" {name}(")
    end = re.search(r" } (template|//|constexpr|__device__)", text[start:])
    return text[start:start + end.start()]


def test_the_second_cta_releases_its_writes_to_the_cluster():
    body = function("clear_tails")
    assert "mbar_arrive_cluster(" not in body
    assert re.search(r"st\.shared.*fence_proxy_async_smem\(\); __syncwarp\(\); if \(lane == 0\) \{ if \(w\.cta == 0\) "
                     r"mbar_arrive\(&w\.sh\.full\[r\.stage\]\); else copy16_to_cluster\(word, at \+ first \* 128, full0 \+ r\.stage \* 8\); \}", body)
    assert "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes" in function("copy16_to_cluster", "tcgen05.cuh")


def test_the_first_cta_waits_for_it():
    """A stage that ends a segment: two arrivals of the first CTA (its loads' issuer, its cleared rows) and 16 bytes."""
    body = function("load_tiles")
    assert re.search(r"if \(w\.ragged\(t, k\)\) \{ bar = [^;]*; mbar_arrive_expect_tx\(&w\.sh\.tail\[r\.stage\], bytes\); "
                     r"if \(w\.cta == 0\) mbar_arrive_expect_tx\(&w\.sh\.full\[r\.stage\], 16\); \}", body)
    assert "mbar_init(&sh.full[i], F == WEIGHTS ? 2 : 1)" in source("matmul_bf16.cu")
