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


def product(a=A, rows=100, k=256, w=B, n=64, E=8, base=C, swiglu=0, out=D, status=None):
    return ep.lib.ep_expert_matmul_bf16(a, rows, k, w, n, E, base, swiglu, out, status, None)


def grad_rows(dc=A, rows=100, n=64, w=B, k=256, E=8, base=C, out=D, status=None):
    return ep.lib.ep_expert_matmul_grad_rows(dc, rows, n, w, k, E, base, out, status, None)


def grad_weights(dc=A, a=B, rows=100, n=64, k=256, E=8, base=C, wide=0, add=0, out=D, status=None):
    return ep.lib.ep_expert_matmul_grad_weights(dc, a, rows, n, k, E, base, wide, add, out, status, None)


SEGMENTS = [dict(rows=-1), dict(rows=(1 << 31) - 1), dict(k=0), dict(k=-8), dict(k=252), dict(k=65544), dict(n=0), dict(n=65537),
            dict(E=0), dict(E=513), dict(base=None), dict(base=C + 2), dict(status=C + 2), dict(out=None), dict(out=D + 1)]


@pytest.mark.parametrize("kw", SEGMENTS + [dict(a=None), dict(a=A + 8), dict(w=None), dict(w=B + 8), dict(n=63, swiglu=1), dict(swiglu=2)])
def test_product_refuses(kw):
    assert product(**kw) == ep.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", SEGMENTS + [dict(dc=None), dict(dc=A + 8), dict(w=None), dict(w=B + 8), dict(n=60), dict(n=4), dict(out=D + 2)])
def test_grad_rows_refuses(kw):
    assert grad_rows(**kw) == ep.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", SEGMENTS + [dict(dc=None), dict(dc=A + 8), dict(a=None), dict(a=B + 8), dict(n=60), dict(n=4), dict(wide=2),
                                           dict(add=2, wide=1), dict(out=D + 2)])
def test_grad_weights_refuses(kw):
    assert grad_weights(**kw) == ep.EP_ERR_INVALID_ARG


def test_sums_of_weights_gradients_are_float32():
    assert grad_weights(add=1) == ep.EP_ERR_UNSUPPORTED


def test_products_of_no_rows():
    assert product(rows=0, a=None, out=None) == ep.EP_OK
    assert grad_rows(rows=0, dc=None, out=None) == ep.EP_OK


def test_binding_refuses_wrong_products():
    f, bf, i4 = torch.zeros, torch.bfloat16, torch.int32
    base = [dict(expert_base=None), dict(expert_base=f(3, dtype=i4)), dict(expert_base=f(4, dtype=torch.int64)),
            dict(expert_base=f(8, dtype=i4)[::2])]
    good = dict(a=f(4, 64, dtype=bf), w=f(3, 32, 64, dtype=bf), expert_base=f(4, dtype=i4), out=f(4, 32, dtype=bf))
    refused(ep.ep_expert_matmul_bf16, good, base + [
        dict(a=f(4, 64)), dict(a=f(64, 4, dtype=bf).t()), dict(a=f(64, dtype=bf)), dict(a=f(4, 128, dtype=bf)[:, ::2]), dict(w=f(3, 32, 64)),
        dict(w=f(3, 32, 48, dtype=bf)), dict(w=f(32, 64, dtype=bf)), dict(w=f(3, 64, 32, dtype=bf).transpose(1, 2)), dict(out=f(4, 32)),
        dict(out=f(4, 16, dtype=bf)), dict(out=f(3, 32, dtype=bf)), dict(swiglu=True)])
    good = dict(grad_c=f(4, 32, dtype=bf), w=good["w"], expert_base=good["expert_base"], grad_a=f(4, 64, dtype=bf))
    refused(ep.ep_expert_matmul_grad_rows, good, base + [
        dict(grad_c=f(4, 32)), dict(grad_c=f(4, 16, dtype=bf)), dict(grad_c=f(32, 4, dtype=bf).t()), dict(w=f(3, 32, 64)),
        dict(grad_a=f(4, 32, dtype=bf)), dict(grad_a=f(4, 64)), dict(grad_a=f(3, 64, dtype=bf))])
    good = dict(grad_c=good["grad_c"], a=f(4, 64, dtype=bf), expert_base=good["expert_base"], grad_w=f(3, 32, 64, dtype=bf))
    refused(ep.ep_expert_matmul_grad_weights, good, base + [
        dict(grad_c=f(3, 32, dtype=bf)), dict(a=f(4, 64)), dict(a=f(64, 4, dtype=bf).t()), dict(grad_w=f(3, 32, 64, dtype=torch.float16)),
        dict(grad_w=f(3, 64, 32, dtype=bf)), dict(grad_w=f(32, 64, dtype=bf)), dict(grad_w=f(3, 64, 32, dtype=bf).transpose(1, 2))])


def fp8(a=A, sa=A, rows=100, k=256, w=B, sw=B, n=64, E=8, base=C, swiglu=0, out=D, status=None):
    return ep.lib.ep_expert_matmul_fp8(a, sa, rows, k, w, sw, n, E, base, swiglu, out, status, None)


@pytest.mark.parametrize("kw", SEGMENTS + [dict(a=None), dict(a=A + 8), dict(w=None), dict(w=B + 8), dict(sa=None), dict(sa=A + 2),
                                           dict(sw=None), dict(sw=B + 2), dict(k=64), dict(k=192), dict(k=65664), dict(n=63, swiglu=1),
                                           dict(swiglu=2)])
def test_fp8_product_refuses(kw):
    assert fp8(**kw) == ep.EP_ERR_INVALID_ARG


def test_fp8_product_of_no_rows():
    assert fp8(rows=0, a=None, sa=None, out=None) == ep.EP_OK


def test_binding_refuses_wrong_fp8_products():
    f, bf, e4 = torch.zeros, torch.bfloat16, torch.float8_e4m3fn
    good = dict(a=f(4, 256, dtype=e4), a_scales=f(4, 2), w=f(3, 320, 256, dtype=e4), w_scales=f(3, 3, 2),
                expert_base=f(4, dtype=torch.int32), out=f(4, 320, dtype=bf))
    bads = [dict(a=f(4, 256, dtype=bf)), dict(a=f(256, 4, dtype=e4).t()), dict(a=f(4, 128, dtype=e4)), dict(a_scales=f(4, 1)),
            dict(a_scales=f(4, 4)[:, ::2]), dict(w=f(3, 320, 256, dtype=torch.uint8)), dict(w=f(3, 256, 320, dtype=e4).transpose(1, 2)),
            dict(w_scales=f(3, 2, 2)), dict(w_scales=f(3, 3, 2, dtype=bf)), dict(expert_base=None), dict(out=f(4, 320)),
            dict(out=f(4, 160, dtype=bf)), dict(swiglu=True), dict(swiglu=True, out=f(4, 160, dtype=bf)),
            dict(a=f(4, 192, dtype=e4), a_scales=f(4, 1), w=f(3, 320, 192, dtype=e4), w_scales=f(3, 3, 1))]
    refused(ep.ep_expert_matmul_fp8, good, bads)


def test_layers_refuse_mixed_weights():
    from combine_ep_layout_03_gb300.expert_layer import ExpertLayer, TrainableExperts
    f, bf, e4, i8 = torch.zeros, torch.bfloat16, torch.float8_e4m3fn, torch.int8
    gamma, s = f(128, dtype=bf), f(4, 2, 1)
    for w13, s13, w2, s2 in ((bf, s, bf, s), (bf, None, bf, s), (e4, None, e4, None), (i8, None, i8, None), (e4, s, i8, s), (bf, None, e4, s)):
        with pytest.raises(ep.EPError) as e:
            ExpertLayer(1, 100, f(4, 256, 128, dtype=w13), s13, f(4, 128, 128, dtype=w2), s2, gamma, 2)
        assert e.value.status == ep.EP_ERR_INVALID_ARG
    with pytest.raises(ep.EPError):   # FP8: whole blocks
        ExpertLayer(1, 100, f(4, 128, 128, dtype=e4), s, f(4, 128, 64, dtype=e4), s, gamma, 2)
    layer = ExpertLayer(1, 8, f(4, 256, 128, dtype=e4), s, f(4, 128, 128, dtype=e4), s, gamma, 2)
    assert not layer.few and layer.rows.dtype is e4
    with pytest.raises(ep.EPError):
        TrainableExperts(1, 0, f(4, 256, 128, dtype=bf), f(4, 128, 128, dtype=bf), 2)
