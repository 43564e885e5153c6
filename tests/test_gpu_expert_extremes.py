"""Expert-layer operators where values leave the range of a type, against the formulas.

The formulas in float32 say which results are infinite, zero or NaN; finite results are compared with
float64.  Sums here are exact (one term, or codes of one size), so what is left is a few float32
roundings, exp and quotient within 2^-20, and the output's own rounding, 2^-8: 2^-7 bounds all of them."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

pytestmark = pytest.mark.gpu


def agrees(got, want, least=0.0):
    """got (bf16) against want (float64 of the float32 formula, where that is finite; else its inf or NaN).
    least: half a step of the smallest bf16, where results are that small."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])
    fine = torch.isfinite(want)
    assert ((got[fine] - want[fine]).abs() <= 2.0 ** -7 * want[fine].abs() + least).all()


def swiglu_of(g, u):
    """silu(g) u by the formula in float32 where that leaves the range, by float64 where not."""
    f = g.float() / (1 + torch.exp(-g.float())) * u.float()
    d = g / (1 + torch.exp(-g)) * u
    return torch.where(torch.isfinite(f) & (f != 0), d, f.double())


@pytest.mark.parametrize("rows,experts", [(4, 1), (300, 1), (600, 2), (40, 16)])
@pytest.mark.parametrize("up_scale", [1e-5, 1e-39])   # 1e-39: the largest gates by the smallest ups
def test_products_with_swiglu(rows, experts, up_scale):
    """Gates and ups of both signs and of 1 to infinity, by each of the kernels that sizes choose."""
    K, half = 128, 72
    sign = torch.where(torch.arange(half, device="cuda") % 2 == 0, 1, -1).to(torch.int8)
    up = torch.where(torch.arange(half, device="cuda") % 3 == 0, 1, -1).to(torch.int8)
    w = torch.cat([sign, up])[None, :, None].expand(experts, 2 * half, K).contiguous()
    sw = torch.ones(experts, 2 * half, device="cuda")
    sw[:, half:] = up_scale
    a = torch.ones(rows, K, dtype=torch.int8, device="cuda")
    sizes = torch.tensor([2.0 ** -7, 0.25, 1e4, 1e20, 1e23, 1e30, 2e36, float("inf")], device="cuda")
    sa = sizes[torch.arange(rows, device="cuda") % len(sizes)].contiguous()
    out = torch.zeros(rows, half, dtype=torch.bfloat16, device="cuda")
    base = torch.linspace(0, rows, experts + 1).int().cuda() if experts > 1 else None
    ep.ep_expert_matmul(a, sa, w, sw, base, out, swiglu=True)
    torch.cuda.synchronize()
    g = K * sa[:, None] * sign.float()
    u = (K * sa[:, None] * up.float()) * sw[0, half:]
    agrees(out, swiglu_of(g.double(), u.double()), 2.0 ** -134)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T,I", [(3, 16), (12, 48), (40, 272)])
@pytest.mark.parametrize("gate,up,weight", [
    (2.0 ** 60, 2.0 ** 80, 1.0),             # an inner value past float32: inf
    (2.0 ** 60, -2.0 ** 80, 1.0),
    (2.0 ** 100, 1.9921875 * 2.0 ** 27, 1.003),    # past the largest bf16, not past float32
    (2.0 ** 100, -1.9921875 * 2.0 ** 27, 1.003),
    (-2.0 ** 60, 2.0 ** 80, 1.0),            # the sigmoid is 0
    (2.0 ** 20, 2.0 ** 30, 1.0),
    (float("inf"), 1.0, 1.0), (1.0, float("-inf"), 1.0), (float("-inf"), 1.0, 1.0)])
def test_inner_values_of_the_few_token_layer(int8, T, I, gate, up, weight):
    """One token has such gates and ups; the others' rows stay as they are without it."""
    H, E = 64, 2
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 1:] = 0
    odd = T // 2
    idx = torch.zeros(T, 1, dtype=torch.int64, device="cuda")
    idx[odd] = 1
    wts = torch.ones(T, 1, device="cuda")
    wts[odd] = weight
    column = torch.where(torch.arange(H, device="cuda") % 2 == 0, 1.0, -1.0)
    ones = torch.zeros(E, 2 * I, H, device="cuda")
    ones[:, :, 0] = 1
    size = torch.ones(E, 2 * I, device="cuda")
    size[1, :I], size[1, I:] = gate, up
    if int8:
        w13, s13 = ones.to(torch.int8), size
        w2, s2 = column.to(torch.int8)[None, :, None].expand(E, H, I).contiguous(), torch.full((E, H), 2.0 ** -20, device="cuda")
    else:
        w13, s13 = (ones * 1).to(torch.bfloat16), None
        w13[:, :, 0] = size.to(torch.bfloat16)
        w2, s2 = (column * 2.0 ** -20)[None, :, None].expand(E, H, I).to(torch.bfloat16).contiguous(), None
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ep.ep_moe_few_tokens_workspace_size(T, H, E, 1, I), dtype=torch.uint8, device="cuda")
    ep.ep_moe_few_tokens(x, idx, wts, w13, w2, out, ws, w13_scales=s13, w2_scales=s2)
    torch.cuda.synchronize()
    assert int8 or torch.equal(w13[1, :, 0].float(), size[1])
    g, u = (torch.tensor(v, dtype=torch.float64, device="cuda") for v in ([1.0, gate], [1.0, up]))
    h = swiglu_of(g, u) * torch.tensor([1.0, weight], device="cuda").double()
    sums = h[idx[:, 0], None] * column.double() * I   # of int8 codes in float32, which the channel's scale then multiplies
    agrees(out, (sums.float().double() if int8 else sums) * 2.0 ** -20)


@pytest.mark.parametrize("rows,empty", [(100, 8), (100, 0), (2000, 0)])
@pytest.mark.parametrize("bases,error", [([0, -5, 50, 100], "order"), ([90, 20, 60, 100], "order"), ([0, 100, 0, 100], "order"),
                                         ([-1, 10, 20, 100], "order"), ([0, 150, 20, 100], "order"), ([0, 50, 101, 101], "rows"),
                                         ([0, 0, 0, 101], "rows"), ([3, 3, 40, 100], None)])
def test_segments_ascend_inside_the_rows(rows, empty, bases, error):
    """Segments that overlap, or lie outside, are an error: nothing is written.  (Empty experts behind them
    make rows an expert few, so that the small product's kernel has its turn.)"""
    f, E = rows // 100, 3 + empty
    bases = bases + bases[-1:] * empty
    base = torch.tensor([b * f if b != 101 else rows + 1 for b in bases], dtype=torch.int32, device="cuda")
    a = torch.ones(rows, 64, dtype=torch.int8, device="cuda")
    w = torch.ones(E, 32, 64, dtype=torch.int8, device="cuda")
    out = torch.full((rows, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ep.ep_expert_matmul(a, torch.ones(rows, device="cuda"), w, torch.ones(E, 32, device="cuda"), base, out, status=status)
    assert status.item() == {None: ep.EP_OK, "order": ep.EP_ERR_INVALID_ARG, "rows": ep.EP_ERR_CAPACITY}[error]
    first = 3 * f if error is None else rows
    assert (out[:first] == 7).all() and (out[first:] == 64).all()


@pytest.mark.parametrize("rows,experts", [(4, 1), (300, 1), (600, 2), (40, 16)])
def test_gates_far_below_zero(rows, experts):
    """Where the sigmoid is near the smallest normal number and the ups are large: products of 1e-6 or so, the
    same of each kernel.  (exp is within 2^-16: 88 log2 e is rounded to float32.)"""
    K, half = 128, 40
    gates = torch.linspace(-88.6, -80, rows, device="cuda")
    a = torch.ones(rows, K, dtype=torch.int8, device="cuda")
    w = torch.ones(experts, 2 * half, K, dtype=torch.int8, device="cuda")
    sw = torch.ones(experts, 2 * half, device="cuda")
    sw[:, half:] = -1e28
    sa = (gates / K).contiguous()
    out = torch.zeros(rows, half, dtype=torch.bfloat16, device="cuda")
    base = torch.linspace(0, rows, experts + 1).int().cuda() if experts > 1 else None
    ep.ep_expert_matmul(a, sa, w, sw, base, out, swiglu=True)
    torch.cuda.synchronize()
    g = (K * sa.double())[:, None].expand(rows, half)
    want = g / (1 + torch.exp(-g)) * (g * sw[0, half:].double())
    assert (want.abs() > 1e-8).all()
    agrees(out, want)
