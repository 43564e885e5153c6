"""SwiGLU with 8-bit checkpoints (ep_swiglu_keep, ep_swiglu_keep_grad) against float64.

Tolerances, from the arithmetic.  The exponential's argument is off by 2^-24 of itself for its rounding and as much for
its constant and (backward) for the rounding of g, so with its own error and the reciprocal's the sigmoid s and
silu = g s are off by a relative eta = (|g| + 8) 2^-22.  Then: inner by (eta + 2^-22) |inner|; g's gradient w dy u
(s + silu (1 - s)) by |w dy u| s eta (1 + 2 |g|) + 2^-22 of itself, since 1 - s is off by eta s + 2^-24; u's by (eta +
2^-22); a weight's gradient by the same of each term and (I / 32 + 8) 2^-24 of their magnitudes' sum for its additions.
Outputs in bf16 add 2^-8 of the value; what the approximations flush to zero, 2^-125 of the factors beside it: a sigmoid
flushed below 2^-126 puts s + g s (1 - s) off by that times 1 + |g|.
Codes are the nearest ones, exactly: a quotient that is no tie is at least 2^-24 away from one."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


def nearest_e4m3(v):
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def make(rows, inner, seed=0, weights=True, scale=1.5, spare=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    total = rows + spare
    c = (torch.randn(total, 2 * inner, device="cuda", generator=g) * scale).to(torch.bfloat16)
    w = torch.rand(total, device="cuda", generator=g) + 0.01 if weights else None
    dy = torch.randn(total, inner, device="cuda", generator=g).to(torch.bfloat16)
    return dict(c=c, w=w, dy=dy, rows=rows, inner=inner, total=total)


def keep(s, used="count", stream=None):
    total, inner = s["total"], s["inner"]
    y = torch.full((total, inner), 7.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((total, 2 * inner), 7.0, device="cuda").to(torch.float8_e4m3fn)
    scales = torch.full((total, inner // 64), 7.0, device="cuda")
    n = torch.tensor([s["rows"]], dtype=torch.int32, device="cuda") if used == "count" else used
    ep.ep_swiglu_keep(s["c"], y, codes, scales, row_weights=s["w"], rows_used=n, stream=stream)
    torch.cuda.synchronize()
    return y, codes, scales


def back(s, codes, scales, used="count", stream=None, inner=True, dweights=True):
    total, I = s["total"], s["inner"]
    dc = torch.full((total, 2 * I), 7.0, dtype=torch.bfloat16, device="cuda")
    y = torch.full((total, I), 7.0, dtype=torch.bfloat16, device="cuda") if inner else None
    dw = torch.full((total,), 7.0, device="cuda") if dweights else None
    n = torch.tensor([s["rows"]], dtype=torch.int32, device="cuda") if used == "count" else used
    ep.ep_swiglu_keep_grad(codes, scales, s["dy"], dc, inner=y, row_weights=s["w"], row_weights_grad=dw, rows_used=n, stream=stream)
    torch.cuda.synchronize()
    return dc, y, dw


def within(got, want, tol):
    worst = ((got.double() - want).abs() - tol).max().item()
    assert worst <= 0, worst


def check_keep(s):
    y, codes, scales = keep(s)
    rows, inner = s["rows"], s["inner"]
    c = s["c"][:rows].double()
    g, u = c.chunk(2, 1)
    wu = u if s["w"] is None else u * s["w"][:rows].double()[:, None]
    z = g * torch.sigmoid(g) * wu
    eta = (g.abs().clamp_max(1e4) + 8) * 2.0 ** -22
    within(y[:rows], z, (eta + 2.0 ** -22 + BF16) * z.abs() + 2.0 ** -125 * (1 + (g * wu).abs()))
    blocks = c.reshape(-1, 128)
    top = blocks.abs().amax(1, keepdim=True)
    assert torch.equal(codes[:rows].double().reshape(-1, 128), nearest_e4m3(blocks * 448 / torch.where(top > 0, top, 1.0)))
    within(scales[:rows].reshape(-1, 1), top / 448, top / 448 * 2.0 ** -24 + 2.0 ** -150)
    for t in (y, codes, scales):
        assert (t[rows:].double() == 7).all()
    return codes, scales


def check_back(s, codes, scales, **kw):
    dc, y, dw = back(s, codes, scales, **kw)
    rows, inner = s["rows"], s["inner"]
    c = codes[:rows].double() * scales[:rows].double().repeat_interleave(128, 1)
    (g, u), dy = c.chunk(2, 1), s["dy"][:rows].double()
    w = 1.0 if s["w"] is None else s["w"][:rows].double()[:, None]
    sig = torch.sigmoid(g)
    silu = g * sig
    eta, tiny = (g.abs().clamp_max(1e4) + 8) * 2.0 ** -22, 2.0 ** -125
    dg, du = w * dy * u * (sig + silu * torch.sigmoid(-g)), w * dy * silu
    within(dc[:rows, :inner], dg, (w * dy * u).abs() * (sig * eta * (1 + 2 * g.abs()) + tiny * (1 + g.abs())) + (2.0 ** -22 + BF16) * dg.abs() + tiny)
    within(dc[:rows, inner:], du, (eta + 2.0 ** -22 + BF16) * du.abs() + tiny * (1 + (w * dy * g).abs()))
    if y is not None:
        z = w * silu * u
        within(y[:rows], z, (eta + 2.0 ** -22 + BF16) * z.abs() + tiny * (1 + (w * g * u).abs()))
    if dw is not None:
        terms = dy * silu * u
        within(dw[:rows], terms.sum(1), (terms.abs() * (eta + 2.0 ** -22 + (inner / 32 + 8) * 2.0 ** -24)).sum(1) + tiny * inner)
    for t in (dc, y, dw):
        assert t is None or (t[rows:].double() == 7).all()


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("inner", [128, 256, 384, 768, 1024, 4096])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 33, 300])
def test_sizes(rows, inner, weights):
    s = make(rows, inner, seed=rows + inner, weights=weights)
    check_back(s, *check_keep(s))


@pytest.mark.parametrize("scale", [1e-37, 1e-30, 1e-3, 30.0, 1e4, 1e18])
def test_ranges(scale):
    """Values from the smallest numbers to ones whose exponential leaves the range."""
    s = make(65, 256, seed=3, scale=scale)
    check_back(s, *check_keep(s))


def test_ties_and_zeros():
    """Quotients on borders between codes (448 c / top with top = 448 or a power of two), zero groups and rows."""
    s = make(64, 128, seed=1)
    c = torch.arange(64 * 256, device="cuda").remainder(1789).view(64, 256).float() / 16
    c[:, 0], c[:, 200] = 448, 512
    c[5], c[6, :128], c[7, 128:] = 0, 0, 0
    s["c"][:64] = c.to(torch.bfloat16)
    codes, scales = check_keep(s)
    assert (scales[5] == 0).all() and (codes[5].double() == 0).all()
    check_back(s, codes, scales)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite_values_stay_in_their_group(bad):
    s = make(20, 256, seed=2)
    y0, codes0, scales0 = keep(s)
    dc0, z0, dw0 = back(s, codes0, scales0)
    s["c"][3, 130] = bad       # a gate of the second group
    y, codes, scales = keep(s)
    assert torch.isnan(scales[3, 1]) and (codes[3, 128:256].double() == 0).all()
    scales[3, 1], codes[3, 128:256] = scales0[3, 1], codes0[3, 128:256]
    assert torch.equal(scales, scales0) and torch.equal(codes.view(torch.uint8), codes0.view(torch.uint8))
    keep_cols = torch.arange(256, device="cuda") != 130
    assert torch.equal(y[:, keep_cols], y0[:, keep_cols])
    scales[3, 1] = float("nan")
    dc, z, dw = back(s, codes, scales)
    assert torch.isnan(dc[3, 128:256]).all() and torch.isnan(z[3, 128:]).all() and torch.isnan(dw[3])
    dc[3], z[3], dw[3] = dc0[3], z0[3], dw0[3]
    assert torch.equal(dc, dc0) and torch.equal(z, z0) and torch.equal(dw, dw0)


@pytest.mark.parametrize("used,rows", [(None, 12), (0, 0), (-5, 0), (5, 5), (12, 12), (99, 12)])
def test_rows_used(used, rows):
    s = make(rows, 128, seed=4, spare=12 - rows)
    n = None if used is None else torch.tensor(used, dtype=torch.int32, device="cuda")
    y, codes, scales = keep(s, used=n)
    assert (y[rows:] == 7).all() and (codes[rows:].double() == 7).all() and (scales[rows:] == 7).all()
    assert rows == 0 or not (y[:rows] == 7).all(1).any()
    dc, z, dw = back(s, codes, scales, used=n)
    assert (dc[rows:] == 7).all() and (z[rows:] == 7).all() and (dw[rows:] == 7).all()
    assert rows == 0 or not (dc[:rows] == 7).all(1).any()


def test_outputs_that_are_not_asked_for():
    s = make(9, 256, seed=5)
    codes, scales = check_keep(s)
    check_back(s, codes, scales, inner=False, dweights=False)
    check_back(s, codes, scales, inner=True, dweights=False)
    check_back(s, codes, scales, inner=False, dweights=True)


def test_gradients_against_differences():
    """The gradient of sum(dy * inner) by central differences of the formula at the kept values."""
    s = make(6, 128, seed=6, scale=1.0, spare=0)
    codes, scales = check_keep(s)
    dc, _, dw = back(s, codes, scales)
    c = codes.double() * scales.double().repeat_interleave(128, 1)

    def loss(c, w):
        g, u = c.chunk(2, 1)
        return (s["dy"].double() * w[:, None] * g * torch.sigmoid(g) * u).sum(1)

    w, h = s["w"].double(), 1e-4
    for col in (0, 17, 127, 128, 255):
        d = torch.zeros_like(c)
        d[:, col] = h
        diff = (loss(c + d, w) - loss(c - d, w)) / (2 * h)
        # differences: h^2 / 6 of the third derivative (below |w dy u|), and the output's rounding
        bound = (w * s["dy"].double()[:, col % 128] * (1 + c[:, (col + 128) % 256].abs())).abs()
        within(dc[:, col], diff, BF16 * diff.abs() + 1e-5 * bound + 1e-6)
    diff = (loss(c, w + h) - loss(c, w - h)) / (2 * h)
    within(dw, diff, 1e-5 * (1 + diff.abs()))


def test_streams_and_graphs():
    s = make(40, 384, seed=7)
    ref, st = keep(s), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    again = keep(s, stream=st)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(ref, again))
    dc, dw = torch.zeros(42, 768, dtype=torch.bfloat16, device="cuda"), torch.zeros(42, device="cuda")
    out = [torch.zeros_like(t) for t in ref]
    n = torch.tensor([40], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_swiglu_keep(s["c"], out[0], out[1], out[2], row_weights=s["w"], rows_used=n)
        ep.ep_swiglu_keep_grad(out[1], out[2], s["dy"], dc, row_weights=s["w"], row_weights_grad=dw, rows_used=n)
    s["c"].copy_(make(40, 384, seed=8)["c"])
    n.fill_(33)
    graph.replay()
    torch.cuda.synchronize()
    s["rows"] = 33
    y, codes, scales = keep(s)
    want_dc, _, want_dw = back(s, codes, scales)
    assert torch.equal(out[0][:33], y[:33]) and torch.equal(dc[:33], want_dc[:33]) and torch.equal(dw[:33], want_dw[:33])
    assert (out[0][33:] == 0).all() and (dc[33:] == 0).all() and (dw[33:] == 0).all()


@pytest.mark.parametrize("rows,inner", [(1216, 640), (1217, 640), (1300, 1024), (1216, 128), (3, 65536)])
def test_rows_by_ctas_and_by_warps(rows, inner):
    s = make(rows, inner, seed=rows)
    check_back(s, *check_keep(s))
    assert torch.equal(back(s, *keep(s)[1:])[2], back(s, *keep(s)[1:])[2])


def test_many_rows():
    s = make(70000, 128, seed=9)
    check_back(s, *check_keep(s))


def test_offsets_past_32_bits():
    """More than 2^31 values: the last rows are those of the rows alone."""
    rows, I, n = 530000, 2176, 40
    s = make(n, I, seed=3, spare=0)
    c = torch.zeros(rows, 2 * I, dtype=torch.bfloat16, device="cuda")
    c[-n:] = s["c"]
    w = torch.ones(rows, device="cuda")
    w[-n:] = s["w"]
    big = dict(c=c, w=w, dy=torch.zeros(rows, I, dtype=torch.bfloat16, device="cuda"), rows=rows, inner=I, total=rows)
    big["dy"][-n:] = s["dy"]
    got, want = keep(big, used=None), keep(s, used=None)
    assert all(torch.equal(a[-n:].view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    grads = back(big, *got[1:], used=None), back(s, *want[1:], used=None)
    for a, b in zip(*grads):
        if a.dim() == 2:
            assert torch.equal(a[-n:], b)
        else:   # sums by warps and by CTAs
            assert ((a[-n:] - b).abs() <= 1e-4 * (1 + b.abs())).all()
    assert (grads[0][0][:-n] == 0).all()
