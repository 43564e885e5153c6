"""Refusals of the FP8 and bf16 expert products, their gradients and SwiGLU with checkpoints: argument errors come
back before any CUDA call, so plain numbers stand in for device addresses here."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

A, B, C, D = (1 << 40), (1 << 41), (1 << 42), (1 << 43)   # never dereferenced


def keep(c=A, w=None, rows=10, inner=256, used=None, y=B, codes=C, scales=D):
    return ep.lib.ep_swiglu_keep(c, w, rows, inner, used, y, codes, scales, None)


def keep_grad(codes=A, scales=B, w=None, dy=C, rows=10, inner=256, used=None, dc=D, y=None, dw=None):
    return ep.lib.ep_swiglu_keep_grad(codes, scales, w, dy, rows, inner, used, dc, y, dw, None)


SIZES = [dict(rows=-1), dict(rows=1 << 31), dict(rows=1 << 30, inner=512), dict(inner=0), dict(inner=64), dict(inner=192),
         dict(inner=65664), dict(inner=-128), dict(w=A + 2), dict(used=A + 1)]


@pytest.mark.parametrize("kw", SIZES + [dict(c=None), dict(c=A + 8), dict(y=None), dict(y=B + 2), dict(codes=None),
                                        dict(codes=C + 8), dict(scales=None), dict(scales=D + 2)])
def test_keep_refuses(kw):
    assert keep(**kw) == ep.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", SIZES + [dict(codes=None), dict(codes=A + 8), dict(scales=None), dict(scales=B + 2), dict(dy=None),
                                        dict(dy=C + 8), dict(dc=None), dict(dc=D + 4), dict(y=A + 8), dict(dw=A + 2)])
def test_keep_grad_refuses(kw):
    assert keep_grad(**kw) == ep.EP_ERR_INVALID_ARG


def test_no_rows_to_keep():
    assert keep(rows=0, c=None, y=None, codes=None, scales=None) == ep.EP_OK
    assert keep_grad(rows=0, codes=None, scales=None, dy=None, dc=None) == ep.EP_OK


def refused(call, good, bads):
    for kw in bads:
        with pytest.raises(ep.EPError) as e:
            call(**{**good, **kw}, stream=0)
        assert e.value.status == ep.EP_ERR_INVALID_ARG, kw


def test_binding_refuses_wrong_rows_to_keep():
    f, bf, e4 = torch.zeros, torch.bfloat16, torch.float8_e4m3fn
    good = dict(c=f(4, 512, dtype=bf), inner=f(4, 256, dtype=bf), codes=f(4, 512, dtype=e4), scales=f(4, 4))
    shared = [dict(codes=f(4, 256, dtype=e4)), dict(codes=f(4, 512, dtype=bf)), dict(codes=f(512, 4, dtype=e4).t()),
              dict(scales=f(4, 2)), dict(scales=f(4, 4, dtype=bf)), dict(scales=f(4, 8)[:, ::2]), dict(row_weights=f(3)),
              dict(row_weights=f(4, dtype=bf)), dict(row_weights=f(8)[::2]), dict(rows_used=f(1)),
              dict(rows_used=f(2, dtype=torch.int32))]
    refused(ep.ep_swiglu_keep, good, shared + [
        dict(c=f(4, 512)), dict(c=f(512, dtype=bf)), dict(c=f(512, 4, dtype=bf).t()), dict(inner=f(4, 128, dtype=bf)),
        dict(inner=f(4, 256)), dict(inner=f(3, 256, dtype=bf)),
        dict(c=f(4, 384, dtype=bf), inner=f(4, 192, dtype=bf), codes=f(4, 384, dtype=e4), scales=f(4, 3))])
    good = dict(codes=good["codes"], scales=good["scales"], grad_inner=good["inner"], grad_c=good["c"])
    refused(ep.ep_swiglu_keep_grad, good, shared + [
        dict(grad_inner=f(4, 256)), dict(grad_inner=f(3, 256, dtype=bf)), dict(grad_c=f(4, 512)), dict(inner=f(4, 512, dtype=bf)),
        dict(grad_c=f(4, 1024, dtype=bf)[:, ::2]), dict(row_weights_grad=f(3)), dict(row_weights_grad=f(4, dtype=bf))])
