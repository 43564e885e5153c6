"""Rows in e4m3 come as such, or as the bytes of a receive buffer: other types of one byte would be read as e4m3, and other
types of the same size as float32 scales, without a word.  (Refused before any CUDA call, so CPU tensors do here.)"""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

bf, e4, u8 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8
CODES = [torch.float8_e5m2, torch.int8, torch.bool]
SCALES = [dict(dtype=torch.int32), dict(dtype=torch.float64, half=True), dict(dtype=bf, double=True), dict(dtype=torch.int8, bytes=True)]


def zeros(*shape, dtype=torch.float32, half=False, double=False, bytes=False):
    """As many bytes as a float32 tensor of this shape has."""
    per = 0.5 if half else 2 if double else 4 if bytes else 1
    return torch.zeros(*shape[:-1], int(shape[-1] * per), dtype=dtype)


def refused(call, **args):
    with pytest.raises(ep.EPError) as err:
        call(**args, stream=0)
    assert err.value.status == ep.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(a=torch.zeros(4, 256, dtype=t)) for t in CODES] + [dict(a_scales=zeros(4, 2, **t)) for t in SCALES])
def test_fp8_product(bad):
    good = dict(a=torch.zeros(4, 256, dtype=e4), a_scales=torch.zeros(4, 2), w=torch.zeros(3, 320, 256, dtype=e4),
                w_scales=torch.zeros(3, 3, 2), expert_base=torch.zeros(4, dtype=torch.int32), out=torch.zeros(4, 320, dtype=bf))
    refused(ep.ep_expert_matmul_fp8, **{**good, **bad})


@pytest.mark.parametrize("bad", [dict(codes=torch.zeros(4, 512, dtype=t)) for t in CODES] + [dict(scales=zeros(4, 4, **t)) for t in SCALES])
def test_kept_rows(bad):
    good = dict(codes=torch.zeros(4, 512, dtype=e4), scales=torch.zeros(4, 4))
    c, inner = torch.zeros(4, 512, dtype=bf), torch.zeros(4, 256, dtype=bf)
    refused(ep.ep_swiglu_keep, c=c, inner=inner, **{**good, **bad})
    refused(ep.ep_swiglu_keep_grad, grad_inner=inner, grad_c=c, **{**good, **bad})


@pytest.mark.parametrize("codes,scales", [(e4, torch.float32), (u8, torch.float32), (u8, u8), (e4, u8)])
def test_no_rows_of_either_type_are_taken(codes, scales):
    """With no rows a call is over after its checks."""
    rows, s = torch.zeros(0, 256, dtype=codes), torch.zeros(0, 8 if scales is u8 else 2, dtype=scales)
    w, base = torch.zeros(3, 320, 256, dtype=e4), torch.zeros(4, dtype=torch.int32)
    ep.ep_expert_matmul_fp8(rows, s, w, torch.zeros(3, 3, 2), base, torch.zeros(0, 320, dtype=bf), stream=0)
    ep.ep_swiglu_keep(torch.zeros(0, 256, dtype=bf), torch.zeros(0, 128, dtype=bf), rows, s, stream=0)
    ep.ep_swiglu_keep_grad(rows, s, torch.zeros(0, 128, dtype=bf), torch.zeros(0, 256, dtype=bf), stream=0)
