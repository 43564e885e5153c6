"""Weights' gradients of segments that end anywhere: rows behind a segment's end are not read, whatever they hold.

A sum of L products is off by L 2^-23 of its terms' magnitudes (additions that cut; products of two bf16 are exact)."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

pytestmark = pytest.mark.gpu

U, NAN = 2.0 ** -23, float("nan")


def rows_of(total, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(total, w, device="cuda", generator=g).to(torch.bfloat16) for w in (n, k)]


def check(d, a, got):
    d, a = d.double(), a.double()
    worst = ((got.double() - d.t() @ a).abs() - (d.shape[0] + 2) * U * (d.abs().t() @ a.abs())).max().item() if d.shape[0] else got.abs().max().item()
    assert worst <= 0, worst   # (NaN is not either)


@pytest.mark.parametrize("n,k", [(8, 8), (264, 72), (136, 520)])
@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_every_length_beside_rows_that_are_not_numbers(n, k, first, bad):
    lengths = list(range(0, 84)) + [127, 128, 129, 143, 191, 192, 193, 255, 256, 257]
    base = torch.tensor([0] + lengths).cumsum(0)
    d, a = rows_of(int(base[-1]), n, k, n + k)
    for e in range(1 - first, len(lengths), 2):   # every other expert's
        d[base[e]:base[e + 1]] = bad
        a[base[e]:base[e + 1]] = bad
    got = torch.full((len(lengths), n, k), 7.0, device="cuda")
    ep.ep_expert_matmul_grad_weights(d, a, base.int().cuda(), got)
    for e in range(first, len(lengths), 2):
        check(d[base[e]:base[e + 1]], a[base[e]:base[e + 1]], got[e])


# one tile whose sum is shared by two and four pairs, tiles of 128 rows and of 256
@pytest.mark.parametrize("E,n,k,each", [(1, 512, 512, 1000), (1, 376, 992, 13920), (4, 2048, 512, 2000), (16, 1408, 1024, 160), (3, 40, 24, 4)])
@pytest.mark.parametrize("over", [0, 1, 3, 4, 7, 8, 11, 15])
@pytest.mark.parametrize("behind", [0, 1, 40])
def test_rows_behind_the_last_segment(E, n, k, each, over, behind):
    end = E * each + over
    d, a = rows_of(end + behind, n, k, over + behind)
    d[end:] = NAN
    a[end:] = NAN
    base = torch.arange(E + 1) * each
    base[-1] = end
    got = torch.full((E, n, k), 7.0, device="cuda")
    ep.ep_expert_matmul_grad_weights(d, a, base.int().cuda(), got)
    for e in range(E):
        check(d[base[e]:base[e + 1]], a[base[e]:base[e + 1]], got[e])
