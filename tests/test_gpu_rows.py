"""8-bit rows of normalised and plain bf16 rows (ep_rms_norm_quant, ep_quant_rows).

The reference is the definition in float64.  int8 and FP8 codes with a largest-magnitude
scale are compared exactly: the quotient t * top / max is settled by integers of at most
23 over 16 bits, so float64 finds every tie.  Scales are float32 results: with at most 32
additions in a thread, 5 across a warp and 32 across warps, the (all positive) sum of
squares is off by (32 + 5 + 32) 2^-24 of itself, its root by half of that, and mean, eps,
root, quotient, product and division round six more times: 2^-24 (69 / 2 + 6) < 41 2^-24.
MX exponents are exact; MX codes may lie one side or the other of a tie that the float32
value of y (41 2^-24 off, plus its own roundings) cannot tell from."""
import numpy as np
import pytest
import torch

import oracle
from combine_ep_layout_03_gb300 import ep

pytestmark = pytest.mark.gpu

TOKEN = {ep.EP_QUANT_INT8_PER_TOKEN: 127.0, ep.EP_QUANT_FP8_E4M3_PER_TOKEN: 448.0,
         ep.EP_QUANT_FP8_E5M2_PER_TOKEN: 57344.0}
GROUP = {ep.EP_QUANT_FP8_E4M3_PER_GROUP: 448.0, ep.EP_QUANT_FP8_E5M2_PER_GROUP: 57344.0}
MX = {ep.EP_QUANT_MXFP8_E4M3: 8, ep.EP_QUANT_MXFP8_E5M2: 15}
MODES = [*TOKEN, *GROUP, *MX]
E5M2 = (ep.EP_QUANT_FP8_E5M2_PER_TOKEN, ep.EP_QUANT_FP8_E5M2_PER_GROUP, ep.EP_QUANT_MXFP8_E5M2)
SCALE_TOL = 41 * 2.0 ** -24


def unit(quant):
    return 128 if quant in GROUP else 32 if quant in MX else 8


def block(quant, H):
    return 128 if quant in GROUP else 32 if quant in MX else H


def step_of(v, e5m2):
    """Distance between neighbouring codes around each |v| (float64)."""
    e = torch.frexp(v).exponent - 1
    return torch.exp2(e.clamp_min(-14 if e5m2 else -6).double() - (2 if e5m2 else 3))


def nearest_fp8(v, e5m2):
    s = step_of(v, e5m2)
    top = 57344.0 if e5m2 else 448.0
    return (torch.round(v / s) * s).clamp(-top, top)


def run(x, res, gamma, eps, quant, keep_h=True, h_out=None):
    rows, H = x.shape
    db, sb = ep.ep_recv_row_bytes(H, quant)
    data = torch.full((rows + 2, db), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + 2, sb), 0x5A, dtype=torch.uint8, device="cuda")
    h = h_out if h_out is not None else torch.empty((rows, H), dtype=torch.bfloat16, device="cuda") if keep_h else None
    ep.ep_rms_norm_quant(x, res, gamma, eps, quant, h, data[:rows], scales[:rows])
    torch.cuda.synchronize()
    assert (data[rows:] == 0x5A).all() and (scales[rows:] == 0x5A).all(), "written past the last row"
    return data[:rows], scales[:rows], h


def decode(data, quant):
    if quant == ep.EP_QUANT_INT8_PER_TOKEN:
        return data.view(torch.int8).double()
    return data.view(torch.float8_e5m2 if quant in E5M2 else torch.float8_e4m3fn).double()


def check(x, res, gamma, eps, quant, data, scales, h):
    rows, H = x.shape
    want_h = x if res is None else (x.float() + res.float()).to(torch.bfloat16)
    if h is not None:
        assert torch.equal(h.view(torch.int16), want_h.view(torch.int16))
    v = want_h.double()
    t = (v * gamma.double()).view(rows, -1, block(quant, H))
    e32 = float(np.float32(eps))
    r = 1 / torch.sqrt(v.square().mean(1) + e32)
    m = t.abs().amax(2)
    codes = decode(data, quant).view(t.shape)
    if quant in MX:
        y = t * r[:, None, None]
        # floor(log2 m r) by squares, so that exact powers of two are told from their neighbours
        k = torch.frexp(m * r[:, None]).exponent.double() - 1
        lhs, rhs = m.square() * H, torch.exp2(2 * k) * (v.square().sum(1) + H * e32)[:, None]
        k = torch.where(lhs < rhs, k - 1, torch.where(lhs >= 4 * rhs, k + 1, k))
        se = torch.where(m > 0, (k - MX[quant]).clamp(-127, 127), -127.0)
        assert torch.equal(scales.double(), se.view(rows, -1) + 127)
        q = y * torch.exp2(-se)[:, :, None]
        top = 57344.0 if quant in E5M2 else 448.0
        q = q.clamp(-top, top)
        assert ((codes - q).abs() <= step_of(q, quant in E5M2) / 2 + 2 * SCALE_TOL * q.abs()).all()
        return
    top = {**TOKEN, **GROUP}[quant]
    q = t * top / torch.where(m > 0, m, 1.0)[:, :, None]
    want = torch.round(q) if quant == ep.EP_QUANT_INT8_PER_TOKEN else nearest_fp8(q, quant in E5M2)
    assert torch.equal(codes, want)
    want_s = m * r[:, None] / top
    got_s = scales.view(torch.float32).double().view(want_s.shape)
    assert ((got_s - want_s).abs() <= SCALE_TOL * want_s).all()


def draw(rows, H, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, H, device="cuda", generator=g) * scale).to(torch.bfloat16)
    res = (torch.randn(rows, H, device="cuda", generator=g) * scale).to(torch.bfloat16)
    gamma = (1 + 0.1 * torch.randn(H, device="cuda", generator=g)).to(torch.bfloat16)
    return x, res, gamma


@pytest.mark.parametrize("quant", MODES)
@pytest.mark.parametrize("rows,H", [(1, 8), (1, 8192), (3, 136), (5, 1024), (700, 2056), (333, 4096), (160, 7168), (400, 8192)])
@pytest.mark.parametrize("add", [False, True])
def test_norm_rows(quant, rows, H, add):
    H = max(H // unit(quant), 1) * unit(quant)
    x, res, gamma = draw(rows, H, seed=rows + H)
    res = res if add else None
    check(x, res, gamma, 1e-6, quant, *run(x, res, gamma, 1e-6, quant))


@pytest.mark.parametrize("rows,H", [(3, 512), (400, 1024), (200, 7168)])
def test_normalised_rows_themselves(rows, H):
    """y_out: float32 y (the root off by at most SCALE_TOL, one product more) rounded to bf16."""
    x, res, gamma = draw(rows, H, seed=rows)
    y = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
    data = torch.empty(rows, H, dtype=torch.int8, device="cuda")
    scales = torch.empty(rows, 1, device="cuda")
    ep.ep_rms_norm_quant(x, res, gamma, 1e-6, ep.EP_QUANT_INT8_PER_TOKEN, None, data, scales, y_out=y)
    v = (x.float() + res.float()).to(torch.bfloat16).double()
    want = v * gamma.double() / torch.sqrt(v.square().mean(1, keepdim=True) + float(np.float32(1e-6)))
    assert ((y.double() - want).abs() <= (2.0 ** -8 + 2 * SCALE_TOL) * want.abs()).all()
    ref = run(x, res, gamma, 1e-6, ep.EP_QUANT_INT8_PER_TOKEN)
    assert torch.equal(data.view(torch.uint8), ref[0]) and torch.equal(scales.view(torch.uint8), ref[1])


@pytest.mark.parametrize("quant", MODES)
def test_zero_rows(quant):
    x = torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda")
    run(x, None, torch.ones(256, dtype=torch.bfloat16, device="cuda"), 1e-6, quant)


@pytest.mark.parametrize("quant", MODES)
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -20, 1.0, 2.0 ** 50])
def test_scales_of_values(quant, scale):
    x, res, gamma = draw(40, 1024, seed=5, scale=scale)
    x[7] = 0
    res[7] = 0          # a row of zeros
    x[9, 1:] = 0
    res[9] = 0          # a single value
    x[11, :512] = 0
    res[11, :512] = 0   # groups and blocks of zeros
    check(x, res, gamma, 1e-6, quant, *run(x, res, gamma, 1e-6, quant))


@pytest.mark.parametrize("quant", MODES)
def test_few_significant_bits_make_ties(quant):
    """Values that are small integers: quotients of them tie often."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-254, 255, (500, 512), device="cuda", generator=g).to(torch.bfloat16)
    x[:250, 0] = 254
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    check(x, None, gamma, 0.0, quant, *run(x, None, gamma, 0.0, quant))


@pytest.mark.parametrize("quant", MX)
def test_block_maximum_on_a_power_of_two(quant):
    """Rows of one magnitude with eps 0: max * root is 1 exactly, and its float32 value may be less."""
    mags = torch.arange(128, 256, device="cuda", dtype=torch.float32)
    x = (mags[:, None] * torch.where(torch.arange(96, device="cuda") % 3 == 0, -1.0, 1.0)).to(torch.bfloat16)
    gamma = torch.ones(96, dtype=torch.bfloat16, device="cuda")
    data, scales, h = run(x, None, gamma, 0.0, quant)
    assert (scales == 127 - MX[quant]).all()
    check(x, None, gamma, 0.0, quant, data, scales, h)


@pytest.mark.parametrize("quant", MX)
@pytest.mark.parametrize("scale", [2.0 ** -80, 2.0 ** -45, 1.0, 2.0 ** 45, 2.0 ** 80])
@pytest.mark.parametrize("rows,H", [(300, 1376), (64, 8192), (1, 64)])
def test_block_codes_are_rounded_once_more_at_most(quant, scale, rows, H):
    """Small integers, whose squares' sum is exact: then only y's own rounding to float32, 2^-24 of it (and
    errors of 2^-40), stands between a code and the nearest one."""
    g = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randint(-7, 8, (rows, H), device="cuda", generator=g).to(torch.bfloat16)
    gamma = ((1 + 0.1 * torch.randn(H, device="cuda", generator=g)) * scale).to(torch.bfloat16)
    data, scales, _ = run(x, None, gamma, 1e-6, quant)
    v = x.double()
    y = (v * gamma.double() / torch.sqrt(v.square().mean(1, keepdim=True) + float(np.float32(1e-6)))).view(rows, -1, 32)
    q = y * torch.exp2(127 - scales.double())[:, :, None]
    top = 57344.0 if quant in E5M2 else 448.0
    q = q.clamp(-top, top)
    codes = decode(data, quant).view(q.shape)
    assert ((codes - q).abs() <= step_of(q, quant in E5M2) / 2 + 1.01 * 2.0 ** -24 * q.abs()).all()


@pytest.mark.parametrize("quant", MODES)
def test_strides_and_in_place(quant):
    wide = draw(64, 1024, seed=3)[0]
    x, res = wide[:, :512], wide[:, 512:]
    gamma = draw(1, 512, seed=4)[2]
    ref = run(x.contiguous(), res.contiguous(), gamma, 1e-6, quant)
    got = run(x, res, gamma, 1e-6, quant)
    for a, b in zip(ref, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    keep = x.clone()
    got = run(x, res, gamma, 1e-6, quant, h_out=res)   # the residual stream, in place
    for a, b in zip(ref[:2], got[:2]):
        assert torch.equal(a, b)
    assert torch.equal(res, ref[2]) and torch.equal(x, keep)


@pytest.mark.parametrize("quant", MODES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite(quant, bad):
    x, res, gamma = draw(6, 512, seed=8)
    ref = run(x, res, gamma, 1e-6, quant)
    x[2, 17] = bad
    data, scales, _ = run(x, res, gamma, 1e-6, quant)
    others = [0, 1, 3, 4, 5]
    assert torch.equal(data[others], ref[0][others]) and torch.equal(scales[others], ref[1][others])
    assert (data[2] == 0).all()
    assert (scales[2] == 255).all() if quant in MX else torch.isnan(scales[2].view(torch.float32)).all()


@pytest.mark.parametrize("quant", MODES)
def test_h_not_kept_other_stream_and_repeat(quant):
    x, res, gamma = draw(50, 1024, seed=9)
    ref = run(x, res, gamma, 1e-6, quant)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    db, sb = ep.ep_recv_row_bytes(1024, quant)
    data = torch.empty(50, db, dtype=torch.uint8, device="cuda")
    scales = torch.empty(50, sb, dtype=torch.uint8, device="cuda")
    ep.ep_rms_norm_quant(x, res, gamma, 1e-6, quant, None, data, scales, stream=st)
    st.synchronize()
    assert torch.equal(data, ref[0]) and torch.equal(scales, ref[1])


@pytest.mark.parametrize("quant", MODES)
@pytest.mark.parametrize("rows,H", [(1, 128), (37, 1024), (300, 4096), (300, 7168)])
def test_quant_rows_are_the_dispatch_encoding(quant, rows, H):
    x = draw(rows, H, seed=rows)[0]
    x[0] = 0
    if rows > 3:
        x[1, 5], x[2, 6], x[3, 7] = float("inf"), float("nan"), -float("inf")
    db, sb = ep.ep_recv_row_bytes(H, quant)
    data = torch.empty(rows, db, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, sb, dtype=torch.uint8, device="cuda")
    ep.ep_quant_rows(x, quant, data, scales)
    # the fused dispatch of the same rows, one expert
    lay = ep.EPLayout(1, rows, H, 1, 1)
    lay.layout(torch.zeros(1, rows, 1, dtype=torch.int64, device="cuda"))
    want, want_s = lay.alloc_recv(quant, rows)
    lay.dispatch(x, quant, want, want_s)
    assert torch.equal(data, want) and torch.equal(scales, want_s)
    fine = torch.isfinite(x.float()).all(1).cpu().numpy()
    bits = x.view(torch.int16).cpu().numpy().view(np.uint16)
    od, os_ = oracle.dispatch(oracle.layout(1, rows, 1, 1, 1, np.zeros((1, rows, 1), np.int64)), bits, quant)
    assert np.array_equal(data.cpu().numpy()[fine], od[fine]) and np.array_equal(scales.cpu().numpy()[fine], os_[fine])
