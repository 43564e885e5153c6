"""Weights' gradients over many rows, against float64: long sums are as exact as short ones.

Terms of one sign, where every cut goes the same way.  The tensor cores take 1024 rows at a time, 16 an instruction, whose 16
exact products and sum so far are cut to the float32 of the largest: off by at most 2^-22 of the sum so far, which is half of
the 1024 rows' on average, so 33 2^-22 of their terms in all (64 / 2 and a first one).  The sums of 1024 rows are added up
in float32, rounding to nearest: 2^-24 of the sum so far each, half of it on average.  An addition to what is there
rounds once more, and so does an output in bf16 (2^-8)."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

pytestmark = pytest.mark.gpu

UNEVEN = [1023, 1024, 1025, 1029, 2048, 2051, 0, 3000, 5000, 64, 1040]


def within(got, terms, rows, extra=0.0):
    tol = 33 * 2.0 ** -22 + ((rows + 1023) // 1024 / 2 + 1) * 2.0 ** -24 + extra
    worst = ((got.double() - terms).abs() - tol * terms).max().item()
    assert worst <= 0, (rows, worst)


@pytest.mark.parametrize("lengths,n,k", [
    (UNEVEN, 264, 136), (UNEVEN, 1400, 1024),            # sums that pairs share, tiles of their own
    ([4096] * 8, 512, 2048), ([16384, 16384], 2048, 1024), ([16387], 72, 4096), ([70001], 256, 256), ([2000] * 4, 2048, 512)])
@pytest.mark.parametrize("out", ["float32", "added", "bf16"])
def test_long_sums(lengths, n, k, out):
    g = torch.Generator(device="cuda").manual_seed(sum(lengths) + n)
    base = torch.tensor([0] + lengths).cumsum(0)
    rows = int(base[-1])
    d, a = (torch.rand(rows + 3, w, device="cuda", generator=g).to(torch.bfloat16) for w in (n, k))
    d[rows:] = float("nan")
    a[rows:] = float("nan")
    before = torch.rand(len(lengths), n, k, device="cuda", generator=g) * 100 if out == "added" else torch.full((len(lengths), n, k), 7.0, device="cuda")
    got = before.clone() if out != "bf16" else before.to(torch.bfloat16)
    ep.ep_expert_matmul_grad_weights(d, a, base.int().cuda(), got, accumulate=out == "added")
    for e, length in enumerate(lengths):
        want = d[base[e]:base[e + 1]].double().t() @ a[base[e]:base[e + 1]].double()
        if out == "added":
            want += before[e].double()
        within(got[e], want, length, 2.0 ** -8 if out == "bf16" else 0.0)


def test_of_both_signs():
    """Cuts towards zero make a sum of random signs small as well.  64 instructions of 2^-22 of the sum so far, at most, whose
    root mean square over 1024 rows is that of the result times sqrt(i / 64): 2/3 of 64 2^-22, and no more for longer sums."""
    g = torch.Generator(device="cuda").manual_seed(0)
    d, a = (torch.randn(2 * 16384, w, device="cuda", generator=g).to(torch.bfloat16) for w in (1024, 2048))
    got = torch.empty(2, 1024, 2048, device="cuda")
    ep.ep_expert_matmul_grad_weights(d, a, torch.tensor([0, 16384, 32768], dtype=torch.int32, device="cuda"), got)
    for e in range(2):
        want = d[16384 * e:16384 * (e + 1)].double().t() @ a[16384 * e:16384 * (e + 1)].double()
        assert (got[e].double() - want).norm() <= 64 * 2 / 3 * 2.0 ** -22 * want.norm()
