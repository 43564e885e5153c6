"""Calls of TrainableExperts that its documentation allows: an expert named twice by a token, a backward pass captured and
replayed before its forward pass, two objects on two streams at a time, forward and backward passes in graphs of their own."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

from test_gpu_expert_training import BF16, Step, formula

pytestmark = pytest.mark.gpu


def test_an_expert_named_twice():
    s = Step(2, 70, 256, 8, 4, 128, 8, seed=11)
    s.idx[:, 1] = s.idx[:, 0]
    s.idx[::3, 3] = s.idx[::3, 0]
    leaves = [t.double().requires_grad_() for t in (s.x, s.wts, s.w13, s.w2)]
    want = formula(s, *leaves)
    want.backward(s.grad.double())
    out, grad_x, grad_wts = s.run()
    assert s.layer.status() == ep.EP_OK and (out.double() - want).norm() <= 4 * BF16 * want.norm()
    for got, leaf in zip((grad_x, grad_wts, s.layer.grad_w13, s.layer.grad_w2), leaves):
        assert (got.double() - leaf.grad).norm() <= 0.12 * leaf.grad.norm()   # (as in test_gpu_expert_training.py)
    hit = (s.idx[:, 0] >= 0)
    assert torch.equal(grad_wts[hit, 0], grad_wts[hit, 1])


def captured(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


def test_a_backward_graph_before_its_forward_graph():
    s, ref = (Step(1, 90, 256, 8, 2, 128, 16, seed=12) for _ in range(2))
    want = ref.run()   # (loads the kernels as well)
    torch.cuda.synchronize()
    forward, out = captured(lambda: s.layer.forward(s.x, s.idx, s.wts))
    backward, (grad_x, grad_wts) = captured(lambda: s.layer.backward(s.grad))
    backward.replay()   # no layout has run: there are no rows
    torch.cuda.synchronize()
    assert (grad_x == 0).all() and (grad_wts == 0).all() and (s.layer.grad_w13 == 0).all() and (s.layer.grad_w2 == 0).all()
    forward.replay()
    backward.replay()
    torch.cuda.synchronize()
    assert s.layer.status() == ep.EP_OK
    assert all(torch.equal(a, b) for a, b in zip((out, grad_x, grad_wts), want))
    assert torch.equal(s.layer.grad_w13, ref.layer.grad_w13) and torch.equal(s.layer.grad_w2, ref.layer.grad_w2)


def test_two_objects_on_two_streams():
    shapes = [(1, 600, 512, 16, 4, 384, 1), (2, 250, 1024, 8, 2, 256, 128)]
    refs = [Step(*a, seed=20 + i) for i, a in enumerate(shapes)]
    wants = [s.run() for s in refs]
    steps = [Step(*a, seed=20 + i) for i, a in enumerate(shapes)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    outs = [None, None]
    for _ in range(8):
        for i, s in enumerate(steps):
            s.layer.zero_grad(streams[i])
            outs[i] = s.run(streams[i])
    torch.cuda.synchronize()
    for s, ref, out, want in zip(steps, refs, outs, wants):
        assert s.layer.status() == ep.EP_OK and all(torch.equal(a, b) for a, b in zip(out, want))
        assert torch.equal(s.layer.grad_w13, ref.layer.grad_w13) and torch.equal(s.layer.grad_w2, ref.layer.grad_w2)
