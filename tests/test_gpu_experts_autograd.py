"""TrainableExperts inside an autograd function, as its module's documentation shows it, and outside of one."""
import re
import textwrap

import pytest
import torch

from combine_ep_layout_03_gb300 import ep, expert_layer

pytestmark = pytest.mark.gpu


def documented():
    """The class of the documentation, and the line that uses it."""
    text = re.search(r"^    class Experts\(.*?^    out = Experts\.apply\([^)]*\)", expert_layer.__doc__, re.S | re.M).group(0)
    *lines, use = textwrap.dedent(text).splitlines()
    scope = {"torch": torch}
    exec("\n".join(lines), scope)
    return scope, use


def test_the_documented_function():
    N, H, E, K, I = 50, 256, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    w13, w2 = (r(E, 2 * I, H) / 16).to(torch.bfloat16), (r(E, H, I) / 11).to(torch.bfloat16)
    x, grad = r(N, H).to(torch.bfloat16).requires_grad_(), r(N, H).to(torch.bfloat16)
    logits = r(N, K).requires_grad_()
    topk_idx = torch.rand(N, E, device="cuda", generator=g).topk(K, 1).indices
    experts = expert_layer.TrainableExperts(1, N, w13, w2, K)
    plain = experts.forward(x, topk_idx, torch.softmax(logits, 1))
    assert not plain.requires_grad
    want_x, want_weights = experts.backward(grad)
    want_w13 = experts.grad_w13.clone()
    scope, use = documented()
    scope.update(x=x, topk_weights=torch.softmax(logits, 1), topk_idx=topk_idx, experts=experts)
    scope["topk_weights"].retain_grad()
    experts.zero_grad()
    exec(use, scope)
    assert torch.equal(scope["out"], plain) and experts.status() == ep.EP_OK
    scope["out"].backward(grad)
    assert torch.equal(x.grad, want_x) and torch.equal(scope["topk_weights"].grad, want_weights) and torch.equal(experts.grad_w13, want_w13)
    assert torch.isfinite(logits.grad).all()
