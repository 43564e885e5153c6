"""Arguments of ExpertLayer's calls on the GPU: shared rows of both shapes on both ways, and streams.

The shared rows' share is checked as the difference to a call without them: out = bf16(s + shared) with
|s| known from the call without them to half a step, 2^-8 of it, so the two differ from the exact sum by
2^-8 |out| + 2^-8 |s| and S + 8 float32 additions, (S + 8) 2^-23 (|s| + sum|shared|)."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep
from combine_ep_layout_03_gb300.expert_layer import ExpertLayer

pytestmark = pytest.mark.gpu


def make(R, T, few, H=512, E=8, K=2, I=128, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w13 = torch.randint(-100, 101, (E, 2 * I, H), device="cuda", generator=g, dtype=torch.int8)
    w2 = torch.randint(-100, 101, (E, H, I), device="cuda", generator=g, dtype=torch.int8)
    s13 = torch.full((E, 2 * I), 0.02 / H ** 0.5, device="cuda")
    s2 = torch.full((E, H), 0.02 / I ** 0.5, device="cuda")
    layer = ExpertLayer(R, T, w13, s13, w2, s2, torch.ones(H, dtype=torch.bfloat16, device="cuda"), K,
                        few_tokens=64 if few else 0)
    assert layer.few == few
    N = R * T
    x = torch.randn(N, H, device="cuda", generator=g).to(torch.bfloat16)
    idx = torch.rand(N, E, device="cuda", generator=g).topk(K, 1).indices
    wts = torch.softmax(torch.randn(N, K, device="cuda", generator=g), 1)
    return layer, x, idx, wts, g


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("R,T,S", [(1, 8, 3), (1, 12, 1), (2, 6, 3), (4, 2, 2)])
@pytest.mark.parametrize("by_rank", [False, True])
def test_shared_rows(few, R, T, S, by_rank):
    layer, x, idx, wts, g = make(R, T, few, seed=S)
    N, H = R * T, layer.H
    layer.norm(x)
    s = layer.experts(idx, wts).clone().double()
    ranks = torch.randn(R, S, T, H, device="cuda", generator=g).to(torch.bfloat16)
    tokens = ranks.transpose(0, 1).reshape(S, N, H)
    out = layer.experts(idx, wts, ranks if by_rank else tokens).double()
    assert layer.status() == ep.EP_OK
    want = s + tokens.double().sum(0)
    tol = 2.0 ** -8 * (out.abs() + s.abs()) + (S + 8) * 2.0 ** -23 * (s.abs() + tokens.double().abs().sum(0))
    assert ((out - want).abs() <= tol).all()


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("handle", [False, True])
def test_shared_rows_on_another_stream(few, handle):
    """Shared rows that have to be reordered, on a stream of the call's own while the current one is busy."""
    layer, x, idx, wts, g = make(2, 6, few, seed=9)
    ranks = torch.randn(2, 3, 6, layer.H, device="cuda", generator=g).to(torch.bfloat16)
    shared = ranks if few else ranks.transpose(0, 1).reshape(3, 12, layer.H)
    layer.norm(x)
    want = layer.experts(idx, wts, shared).clone()
    layer.out.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)   # a tenth of a second of the current stream
    layer.experts(idx, wts, shared, stream=side.cuda_stream if handle else side)
    side.synchronize()
    with torch.cuda.stream(side):
        got = layer.out.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("few", [False, True])
def test_status_is_that_of_the_last_step(few):
    layer, x, idx, wts, _ = make(1, 8, few, seed=4)
    layer.norm(x)
    bad = idx.clone()
    bad[3, 1] = layer.E
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side):
        for routing, want in ((idx, ep.EP_OK), (bad, ep.EP_ERR_BAD_EXPERT_ID), (idx, ep.EP_OK)):
            layer.experts(routing, wts, stream=stream)
            assert layer.status(stream) == want


@pytest.mark.parametrize("few", [False, True])
def test_status_of_a_captured_step_is_that_of_its_replays(few):
    layer, x, idx, wts, _ = make(1, 8, few, seed=5)
    layer.norm(x)
    want, routing = layer.experts(idx, wts).clone(), idx.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.experts(routing, wts)
    for bad, error in ((False, ep.EP_OK), (True, ep.EP_ERR_BAD_EXPERT_ID), (False, ep.EP_OK)):
        routing.copy_(idx)
        if bad:
            routing[3, 1] = layer.E
        graph.replay()
        assert layer.status() == error
    assert torch.equal(layer.out, want)
