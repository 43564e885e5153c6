"""The expert layer as a whole (expert_layer.ExpertLayer): its steps against float64 of what
each step was given, and its two ways against the unquantised layer.

The long way's bound: each stage is compared with float64 of the very codes and scales that it
read, so only its own arithmetic counts: products round once to bf16 (2^-8; the sums here stay
below 2^24 and are exact), the combine adds K terms and rounds once more.  Against the layer
without 8-bit activations the error is that of two quantisations: a code is off by at most half a
step, amax / 254, evenly spread, so with amax at most 6 rms the rms error of a row is below
6 / 254 / sqrt(3) < 0.014 of its rms for each; the inner row's passes through SwiGLU's products at
most doubled.  0.06 bounds the relative 2-norm."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep
from combine_ep_layout_03_gb300.expert_layer import ExpertLayer

pytestmark = pytest.mark.gpu


def make(R, T, H, E, K, I, alpha, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    w13 = (r(E, 2 * I, H) * 30).round().clamp(-127, 127).to(torch.int8)
    w2 = (r(E, H, I) * 30).round().clamp(-127, 127).to(torch.int8)
    s13 = (torch.rand(E, 2 * I, device="cuda", generator=g) + 0.5) / 30 / H ** 0.5
    s2 = (torch.rand(E, H, device="cuda", generator=g) + 0.5) / 30 / I ** 0.5
    gamma = (1 + 0.1 * r(H)).to(torch.bfloat16)
    layer = ExpertLayer(R, T, w13, s13, w2, s2, gamma, K, alpha=alpha)
    x, res = r(R * T, H).to(torch.bfloat16), r(R * T, H).to(torch.bfloat16)
    idx = torch.rand(R * T, E, device="cuda", generator=g).topk(K, 1).indices
    wts = torch.softmax(r(R * T, K), 1)
    return layer, x, res, idx, wts


def plain(layer, y, idx, wts):
    """The layer in float64 on rows y, activations unquantised."""
    out = torch.zeros(y.shape, dtype=torch.float64, device="cuda")
    for e in range(layer.E):
        hit = idx == e
        t = hit.any(1).nonzero()[:, 0]
        if not len(t):
            continue
        w = torch.where(hit, wts.double(), 0.0).sum(1)[t]
        w13 = layer.w13[e].double() * layer.w13_scales[e].double()[:, None]
        w2 = layer.w2[e].double() * layer.w2_scales[e].double()[:, None]
        g, u = (y[t].double() @ w13.t()).chunk(2, 1)
        out[t] += w[:, None] * ((g * torch.sigmoid(g) * u) @ w2.t())
    return out


@pytest.mark.parametrize("R,T,H,E,K,I,alpha", [(1, 200, 512, 8, 2, 256, 1), (2, 300, 1024, 16, 4, 384, 128),
                                               (4, 33, 256, 64, 8, 128, 16)])
def test_the_long_way(R, T, H, E, K, I, alpha):
    layer, x, res, idx, wts = make(R, T, H, E, K, I, alpha)
    y = layer.norm(x, res)
    assert torch.equal(layer.h, (x.float() + res.float()).to(torch.bfloat16))
    out = layer.experts(idx.view(R, T, K), wts.view(R, T, K)).clone()
    assert layer.status() == ep.EP_OK and not layer.few
    # each stage on its own inputs
    v = layer.layout.views()
    dst, base = v["dst_row"].view(-1, K).long(), v["expert_base"].tolist()
    codes = layer.recv.view(torch.int8)
    assert torch.equal(codes[dst], layer.rows[:, None].expand(-1, K, -1))
    recv = codes.double() * layer.recv_scales.view(torch.float32).double()
    inner = layer.inner_rows.double() * layer.inner_scales.double()
    for e in range(E):
        r = slice(base[e], base[e + 1])
        g, u = (recv[r] @ layer.w13[e].double().t() * layer.w13_scales[e].double()).chunk(2, 1)
        want = g * torch.sigmoid(g) * u
        assert ((layer.inner[r].double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-30).all()
        want = inner[r] @ layer.w2[e].double().t() * layer.w2_scales[e].double()
        assert ((layer.expert_out[r].double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-30).all()
    terms = layer.expert_out[dst].double() * wts.double()[:, :, None]
    bound = 2.0 ** -8 * terms.sum(1).abs() + (2 * K + 1) * 2.0 ** -24 * terms.abs().sum(1)
    assert ((out.double() - terms.sum(1)).abs() <= bound).all()
    # and the whole against the layer without 8-bit activations
    want = plain(layer, y, idx, wts)
    assert (out.double() - want).norm() <= 0.06 * want.norm()


@pytest.mark.parametrize("R,T", [(1, 1), (1, 7), (2, 32), (8, 4)])
def test_the_short_way(R, T):
    layer, x, res, idx, wts = make(R, T, 512, 16, 4, 256, 1, seed=T)
    shared = torch.randn(R, 2, T, 512, device="cuda").to(torch.bfloat16)
    y = layer.norm(x, res)
    out = layer.experts(idx.view(R, T, 4), wts.view(R, T, 4), shared).double()
    assert layer.status() == ep.EP_OK and layer.few
    want = plain(layer, y, idx, wts) + shared.double().sum(1).reshape(R * T, 512)
    assert (out - want).norm() <= 2.0 ** -8 * want.norm()   # every value is within half a step, 2^-8 of it


def test_the_way_is_the_callers_choice():
    layer, x, res, idx, wts = make(1, 40, 512, 16, 4, 256, 1, seed=3)
    assert layer.few
    other = ExpertLayer(1, 40, layer.w13, layer.w13_scales, layer.w2, layer.w2_scales, layer.gamma, topk=4, few_tokens=16)
    assert not other.few
    y = other.norm(x, res)
    assert torch.equal(y, layer.norm(x, res))
    out = other.experts(idx.view(1, 40, 4), wts.view(1, 40, 4)).double()
    assert other.status() == ep.EP_OK
    want = plain(other, y, idx, wts)
    assert (out - want).norm() <= 0.06 * want.norm()
