"""Refusals of the expert-layer operators: argument errors come back before any CUDA
call, so plain numbers stand in for device addresses here."""
import ctypes

import pytest
import torch

from combine_ep_layout_03_gb300 import ep

A, B, C, D = (1 << 40), (1 << 41), (1 << 42), (1 << 43)   # never dereferenced
NAN = float("nan")


def norm(x=A, xs=512, res=None, rs=0, gamma=B, eps=1e-6, rows=4, hidden=512, quant=ep.EP_QUANT_INT8_PER_TOKEN, h=None,
         hs=0, y=None, data=C, scales=D):
    return ep.lib.ep_rms_norm_quant(x, xs, res, rs, gamma, eps, rows, hidden, quant, h, hs, y, data, scales, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=A + 2), dict(xs=504), dict(xs=513), dict(res=A + 4, rs=512), dict(res=A, rs=511),
    dict(res=A, rs=256), dict(gamma=None), dict(gamma=B + 8), dict(eps=-1.0), dict(eps=NAN), dict(rows=-1),
    dict(rows=1 << 31), dict(hidden=0), dict(hidden=500, xs=504), dict(hidden=8200, xs=8200), dict(h=A + 2, hs=512),
    dict(h=A, hs=500), dict(y=A + 8), dict(data=None), dict(data=C + 8), dict(scales=None), dict(scales=D + 2),
    dict(quant=ep.EP_QUANT_FP8_E4M3_PER_GROUP, hidden=192, xs=192), dict(quant=ep.EP_QUANT_MXFP8_E5M2, hidden=48, xs=48)])
def test_norm_refuses(kw):
    assert norm(**kw) == ep.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("quant", [ep.EP_QUANT_NONE, ep.EP_QUANT_INT8_STATIC, ep.EP_QUANT_MXFP4_E2M1, 3, 11, -1])
def test_norm_refuses_other_modes(quant):
    assert norm(quant=quant) == ep.EP_ERR_UNSUPPORTED
    assert ep.lib.ep_quant_rows(A, 512, 4, 512, quant, C, D, None) == ep.EP_ERR_UNSUPPORTED


def test_no_rows_is_fine():
    assert norm(rows=0, x=None, data=None, scales=None) == ep.EP_OK
    assert ep.lib.ep_quant_rows(None, 512, 0, 512, ep.EP_QUANT_INT8_PER_TOKEN, None, None, None) == ep.EP_OK


def test_quant_rows_refuses():
    q = ep.EP_QUANT_INT8_PER_TOKEN
    for args in ((None, 512, 4, 512, q, C, D), (A, 500, 4, 512, q, C, D), (A, 512, -1, 512, q, C, D),
                 (A, 512, 4, 512, q, None, D), (A, 512, 4, 512, q, C, None)):
        assert ep.lib.ep_quant_rows(*args, None) == ep.EP_ERR_INVALID_ARG


def few(x=A, idx=A, wts=A, T=4, H=256, E=8, K=2, I=64, w13=B, s13=None, w2=C, s2=None, shared=None, S=0, out=D, ws=D,
        n=None, status=None):
    n = max(T, 0) * K * I * 4 if n is None else n
    return ep.lib.ep_moe_few_tokens(x, idx, wts, T, H, E, K, I, w13, s13, w2, s2, shared, S, out, ws, n, status, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=A + 8), dict(idx=None), dict(idx=A + 4), dict(wts=None), dict(T=-1), dict(H=252), dict(H=0),
    dict(H=8200), dict(E=0), dict(E=513), dict(K=0), dict(K=9), dict(K=17, E=32), dict(I=4), dict(I=60), dict(I=65544),
    dict(w13=None), dict(w13=B + 8), dict(w2=None), dict(w2=C + 2), dict(s13=B), dict(s2=B),
    dict(s13=B, s2=B, H=264), dict(s13=B, s2=B, I=72), dict(s13=B + 2, s2=B), dict(S=1), dict(S=17, shared=A),
    dict(S=-1), dict(out=None), dict(ws=None), dict(ws=D + 8), dict(n=4 * 2 * 64 * 4 - 1), dict(status=A + 2)])
def test_few_tokens_refuses(kw):
    assert few(**kw) == ep.EP_ERR_INVALID_ARG


def test_few_tokens_limits():
    assert few(T=65) == ep.EP_ERR_UNSUPPORTED
    assert few(T=0, x=None, idx=None, wts=None, out=None, ws=None) == ep.EP_OK
    assert ep.ep_moe_few_tokens_workspace_size(64, 8192, 512, 16, 2048) == 64 * 16 * 2048 * 4
    with pytest.raises(ep.EPError) as e:
        ep.ep_moe_few_tokens_workspace_size(65, 256, 8, 2, 64)
    assert e.value.status == ep.EP_ERR_UNSUPPORTED
    n = ctypes.c_size_t(0)
    assert ep.lib.ep_moe_few_tokens_workspace_size(4, 256, 8, 2, 64, None) == ep.EP_ERR_INVALID_ARG
    assert ep.lib.ep_moe_few_tokens_workspace_size(4, 250, 8, 2, 64, ctypes.byref(n)) == ep.EP_ERR_INVALID_ARG


def matmul(a=A, sa=A, rows=100, k=256, w=B, sw=B, n=64, E=8, base=C, swiglu=0, out=D, status=None):
    return ep.lib.ep_expert_matmul(a, sa, rows, k, w, sw, n, E, base, swiglu, out, status, None)


@pytest.mark.parametrize("kw", [
    dict(a=None), dict(a=A + 8), dict(sa=None), dict(sa=A + 2), dict(rows=-1), dict(rows=(1 << 31) - 1), dict(k=0),
    dict(k=8), dict(k=264), dict(k=65552), dict(w=None), dict(w=B + 8), dict(sw=None), dict(sw=B + 1), dict(n=0),
    dict(n=65537), dict(n=63, swiglu=1), dict(swiglu=2), dict(E=0), dict(E=513), dict(base=None), dict(base=C + 2),
    dict(out=None), dict(out=D + 1), dict(status=C + 2)])
def test_matmul_refuses(kw):
    assert matmul(**kw) == ep.EP_ERR_INVALID_ARG


def test_matmul_of_no_rows():
    assert matmul(rows=0, a=None, sa=None, out=None) == ep.EP_OK


def test_binding_refuses_wrong_tensors():
    """Types, shapes and layouts that a pointer does not show."""
    bf, q = torch.bfloat16, ep.EP_QUANT_INT8_PER_TOKEN
    x, gamma = torch.zeros(4, 64, dtype=bf), torch.zeros(64, dtype=bf)
    data, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    bad = [dict(x=x.float()), dict(x=torch.zeros(64, 4, dtype=bf).t()), dict(res=torch.zeros(3, 64, dtype=bf)),
           dict(gamma=gamma[:32]), dict(gamma=gamma.float()), dict(data=data[:3]), dict(data=data.t()),
           dict(scales=scales[:, :2]), dict(h=torch.zeros(4, 64))]
    for kw in bad:
        a = {**dict(x=x, res=None, gamma=gamma, h=None, data=data, scales=scales), **kw}
        with pytest.raises(ep.EPError) as e:
            ep.ep_rms_norm_quant(a["x"], a["res"], a["gamma"], 1e-6, q, a["h"], a["data"], a["scales"], stream=0)
        assert e.value.status == ep.EP_ERR_INVALID_ARG
    good = dict(x=x, topk_idx=torch.zeros(4, 2, dtype=torch.int64), topk_weights=torch.zeros(4, 2),
                w13=torch.zeros(3, 32, 64, dtype=bf), w2=torch.zeros(3, 64, 16, dtype=bf), out=torch.zeros(4, 64, dtype=bf),
                workspace=torch.zeros(1 << 14, dtype=torch.uint8))
    f = torch.zeros
    for kw in (dict(x=x.float()), dict(topk_idx=f(4, 2, dtype=torch.int32)), dict(topk_weights=f(4, 3)),
               dict(w13=f(3, 32, 64)), dict(w13=f(3, 32, 48, dtype=bf)), dict(w2=f(3, 16, 64, dtype=bf)),
               dict(out=f(4, 64)), dict(shared=f(1, 3, 64, dtype=bf)), dict(w13_scales=f(3, 32)),
               dict(w13=f(3, 32, 64, dtype=torch.int8), w2=f(3, 64, 16, dtype=torch.int8), w13_scales=f(3, 32)),
               dict(w13=f(3, 32, 64, dtype=torch.int8), w2=f(3, 64, 16, dtype=torch.int8), w13_scales=f(3, 31),
                    w2_scales=f(3, 64))):
        with pytest.raises(ep.EPError) as e:
            ep.ep_moe_few_tokens(**{**good, **kw}, stream=0)
        assert e.value.status == ep.EP_ERR_INVALID_ARG
    mm = dict(a=f(4, 64, dtype=torch.int8), a_scales=f(4), w=f(3, 32, 64, dtype=torch.int8), w_scales=f(3, 32),
              expert_base=f(4, dtype=torch.int32), out=f(4, 32, dtype=bf))
    for kw in (dict(a=f(4, 64)), dict(a=f(64, 4, dtype=torch.int8).t()), dict(a_scales=f(3)), dict(w=f(3, 32, 64)),
               dict(w=f(3, 32, 48, dtype=torch.int8)), dict(w_scales=f(32)), dict(expert_base=None),
               dict(expert_base=f(3, dtype=torch.int32)), dict(expert_base=f(4, dtype=torch.int64)),
               dict(out=f(4, 32)), dict(out=f(4, 16, dtype=bf)), dict(swiglu=True)):
        with pytest.raises(ep.EPError) as e:
            ep.ep_expert_matmul(**{**mm, **kw}, stream=0)
        assert e.value.status == ep.EP_ERR_INVALID_ARG
