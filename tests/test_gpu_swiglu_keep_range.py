"""SwiGLU's backward pass where gate times up passes the range of float32 and its weight brings the result back: the
inner rows that it makes again are the formula's, as the forward pass's are.  Tolerances are those of
test_gpu_swiglu_keep.py."""
import pytest
import torch

from test_gpu_swiglu_keep import back, check_back, check_keep, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,inner", [(20, 128), (20, 384), (9, 2048), (1300, 640)])
@pytest.mark.parametrize("scale,weight", [(2e19, 0.01), (6e19, 0.0005)])
def test_gate_times_up_past_the_range(rows, inner, scale, weight):
    s = make(rows, inner, seed=rows, scale=scale)
    s["w"].mul_(weight)
    codes, scales = check_keep(s)
    g, u = s["c"].float().chunk(2, 1)
    assert torch.isinf(g * u).any()
    check_back(s, codes, scales, dweights=False)
    y = back(s, codes, scales, dweights=False)[1]
    assert torch.isfinite(y[:rows].float()).all()
