"""Rows of ep_rms_norm_quant whose squares leave the range of float32, against the definition in float64:
codes, exponents and scales as exact as those of ordinary rows (test_gpu_rows.check), and y itself."""
import numpy as np
import pytest
import torch

from combine_ep_layout_03_gb300 import ep
from test_gpu_rows import GROUP, MODES, MX, SCALE_TOL, check, draw, run

pytestmark = pytest.mark.gpu


def y_of(x, res, gamma, eps):
    rows, H = x.shape
    y = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
    data, scales = torch.empty(rows, H, dtype=torch.int8, device="cuda"), torch.empty(rows, 1, device="cuda")
    ep.ep_rms_norm_quant(x, res, gamma, eps, ep.EP_QUANT_INT8_PER_TOKEN, None, data, scales, y_out=y)
    torch.cuda.synchronize()
    return y


def check_y(x, res, gamma, eps):
    v = (x if res is None else (x.float() + res.float()).to(torch.bfloat16)).double()
    want = v * gamma.double() / torch.sqrt(v.square().mean(1, keepdim=True) + float(np.float32(eps)))
    # 2^-134: half a step of the smallest bf16
    assert ((y_of(x, res, gamma, eps).double() - want).abs() <= (2.0 ** -8 + 2 * SCALE_TOL) * want.abs() + 2.0 ** -134).all()


@pytest.mark.parametrize("quant", MODES)
@pytest.mark.parametrize("eps", [0.0, 1e-38])
@pytest.mark.parametrize("scale", [2.0 ** -124, 2.0 ** -110, 2.0 ** -100, 2.0 ** -76, 2.0 ** -74, 2.0 ** -62, 2.0 ** -50, 2.0 ** -40])
@pytest.mark.parametrize("rows,H", [(5, 1024), (400, 4096), (300, 384)])
@pytest.mark.parametrize("keep_h", [False, True])
def test_rows_of_tiny_values(quant, eps, scale, rows, H, keep_h):
    x, res, gamma = draw(rows, H, seed=rows, scale=scale)
    check(x, res, gamma, eps, quant, *run(x, res, gamma, eps, quant, keep_h))
    check_y(x, res, gamma, eps)


@pytest.mark.parametrize("quant", MODES)
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("scale", [2.0 ** 56, 2.0 ** 58, 2.0 ** 60, 2.0 ** 63, 2.0 ** 64, 2.0 ** 100, 2.0 ** 123])
@pytest.mark.parametrize("rows,H", [(5, 1024), (400, 4096), (300, 384)])
def test_rows_of_huge_values(quant, eps, scale, rows, H):
    x, res, gamma = draw(rows, H, seed=rows, scale=scale)
    x[0], res[0] = x[0] * 2.0 ** -123, res[0] * 2.0 ** -123   # beside an ordinary row
    check(x, None, gamma, eps, quant, *run(x, None, gamma, eps, quant))
    check(x, res, gamma, eps, quant, *run(x, res, gamma, eps, quant))
    check_y(x, res, gamma, eps)


@pytest.mark.parametrize("quant", MODES)
def test_in_place_and_without_a_residual(quant):
    x, res, gamma = draw(50, 1024, seed=2, scale=2.0 ** -90)
    ref = run(x, res, gamma, 0.0, quant)
    got = run(x, res, gamma, 0.0, quant, h_out=res)
    for a, b in zip(ref, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    check(x, None, gamma, 0.0, quant, *run(x, None, gamma, 0.0, quant, False))


@pytest.mark.parametrize("quant", MX)
@pytest.mark.parametrize("power", [-126, -110, -80, 70, 119])
def test_block_maximum_on_a_power_of_two(quant, power):
    """As for ordinary rows: max * root is 1 exactly, and its float32 value may be less."""
    mags = torch.arange(128, 256, device="cuda", dtype=torch.float64) * 2.0 ** power
    x = (mags[:, None] * torch.where(torch.arange(96, device="cuda") % 3 == 0, -1.0, 1.0)).to(torch.bfloat16)
    gamma = torch.ones(96, dtype=torch.bfloat16, device="cuda")
    data, scales, h = run(x, None, gamma, 0.0, quant)
    assert (scales == 127 - MX[quant]).all()
    check(x, None, gamma, 0.0, quant, data, scales, h)


@pytest.mark.parametrize("quant", MODES)
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_zeros(quant, eps):
    """Zero codes, scale 0 (byte 0) and zeros in y, whatever eps; the rows beside them as they are alone."""
    x, res, gamma = draw(40, 512, seed=1)
    x[::3] = 0
    data, scales, _ = run(x, None, gamma, eps, quant)
    assert (data[::3] == 0).all() and (scales[::3] == 0).all()
    y = y_of(x, None, gamma, eps)
    assert (y[::3] == 0).all()
    keep = torch.arange(40, device="cuda") % 3 != 0
    check(x[keep], None, gamma, eps, quant, data[keep], scales[keep], None)


@pytest.mark.parametrize("quant", MODES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_among_huge_values(quant, bad):
    x, _, gamma = draw(6, 512, seed=8, scale=2.0 ** 100)
    ref = run(x, None, gamma, 1e-6, quant)
    x[2, 17] = bad
    data, scales, _ = run(x, None, gamma, 1e-6, quant)
    others = [0, 1, 3, 4, 5]
    assert torch.equal(data[others], ref[0][others]) and torch.equal(scales[others], ref[1][others])
    assert (data[2] == 0).all()
    assert (scales[2] == 255).all() if quant in MX else torch.isnan(scales[2].view(torch.float32)).all()
    y = y_of(x, None, gamma, 1e-6)[2]
    assert torch.isnan(y[17])
    y = torch.cat([y[:17], y[18:]])
    assert torch.isnan(y).all() if bad != bad else (y == 0).all()   # the formula: a number by inf is 0
