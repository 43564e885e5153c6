"""Expert-layer operators where values leave the range of a type, against the formulas.

The formulas in float32 say which results are infinite, zero or NaN; finite results are compared with
float64.  Sums here are exact (one term, or codes of one size), so what is left is a few float32
roundings, exp and quotient within 2^-20, and the output's own rounding, 2^-8: 2^-7 bounds all of them."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

pytestmark = pytest.mark.gpu


def agrees(got, want):
    """got (bf16) against want (float64 of the float32 formula, where that is finite; else its inf or NaN)."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])
    fine = torch.isfinite(want)
    assert ((got[fine] - want[fine]).abs() <= 2.0 ** -7 * want[fine].abs()).all()


def swiglu_of(g, u):
    """silu(g) u by the formula in float32 where that leaves the range, by float64 where not."""
    f = g.float() / (1 + torch.exp(-g.float())) * u.float()
    d = g / (1 + torch.exp(-g)) * u
    return torch.where(torch.isfinite(f) & (f != 0), d, f.double())


@pytest.mark.parametrize("rows,experts", [(4, 1), (300, 1), (600, 2), (40, 16)])
def test_products_with_swiglu(rows, experts):
    """Gates and ups of both signs and of 1 to infinity, by each of the kernels that sizes choose."""
    K, half = 128, 72
    sign = torch.where(torch.arange(half, device="cuda") % 2 == 0, 1, -1).to(torch.int8)
    up = torch.where(torch.arange(half, device="cuda") % 3 == 0, 1, -1).to(torch.int8)
    w = torch.cat([sign, up])[None, :, None].expand(experts, 2 * half, K).contiguous()
    sw = torch.ones(experts, 2 * half, device="cuda")
    sw[:, half:] = 1e-5
    a = torch.ones(rows, K, dtype=torch.int8, device="cuda")
    sizes = torch.tensor([2.0 ** -7, 0.25, 1e4, 1e20, 1e23, 1e30, float("inf")], device="cuda")
    sa = sizes[torch.arange(rows, device="cuda") % len(sizes)].contiguous()
    out = torch.zeros(rows, half, dtype=torch.bfloat16, device="cuda")
    base = torch.linspace(0, rows, experts + 1).int().cuda() if experts > 1 else None
    ep.ep_expert_matmul(a, sa, w, sw, base, out, swiglu=True)
    torch.cuda.synchronize()
    g = K * sa[:, None] * sign.float()
    u = (K * sa[:, None] * up.float()) * sw[0, half:]
    agrees(out, swiglu_of(g.double(), u.double()))
