"""What TrainableExperts hands to the library and when it refuses to, on the CPU: its tensors are CPU tensors here, and the
library's calls are replaced by ones that keep their names."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep
from combine_ep_layout_03_gb300.expert_layer import TrainableExperts

E, H, I, K, N = 4, 64, 128, 2, 6
LAYOUT = ("layout", "dispatch", "expert_matmul_bf16", "expert_matmul_grad_rows", "expert_matmul_grad_weights", "combine")


def weights(E=E, H=H, I=I):
    return torch.zeros(E, 2 * I, H, dtype=torch.bfloat16), torch.zeros(E, H, I, dtype=torch.bfloat16)


def make(monkeypatch):
    """Experts of N tokens, the list that their calls fill, and a set of calls that shall fail."""
    layer, calls, fails = TrainableExperts(1, N, *weights(), K), [], set()

    def keep(name):
        def call(*args, **kw):
            calls.append(name)
            if name in fails:
                raise ep.EPError(ep.EP_ERR_CUDA, name)
            return torch.zeros(N, H, dtype=torch.bfloat16) if name == "combine" else None
        return call

    for name in LAYOUT:
        monkeypatch.setattr(layer.layout, name, keep(name))
    for name in ("ep_swiglu_keep", "ep_swiglu_keep_grad"):
        monkeypatch.setattr(ep, name, keep(name))
    return layer, calls, fails


def step(**other):
    args = dict(x=torch.zeros(N, H, dtype=torch.bfloat16), topk_idx=torch.zeros(N, K, dtype=torch.int64), topk_weights=torch.zeros(N, K))
    return {**args, **other}


GRAD = torch.zeros(N, H, dtype=torch.bfloat16)


def refused(layer, calls):
    """backward() raises, and nothing of the library is called."""
    calls.clear()
    with pytest.raises(ep.EPError) as err:
        layer.backward(GRAD)
    assert err.value.status == ep.EP_ERR_INVALID_ARG and not calls


def test_backward_needs_a_forward(monkeypatch):
    """The layout that backward() moves rows by is memory as it was found until a forward() has written it."""
    layer, calls, _ = make(monkeypatch)
    refused(layer, calls)
    layer.forward(**step())
    calls.clear()
    for _ in range(2):   # of the last forward(), as often as asked for
        grad_x, grad_weights = layer.backward(GRAD)
        assert grad_x.shape == (N, H) and grad_weights.shape == (N, K)
    assert calls.count("dispatch") == 2


@pytest.mark.parametrize("failing", [name for name in LAYOUT if "grad" not in name] + ["ep_swiglu_keep"])
def test_backward_needs_a_whole_forward(failing, monkeypatch):
    """A forward() that stopped on its way has overwritten what the one before it left."""
    layer, calls, fails = make(monkeypatch)
    layer.forward(**step())
    fails.add(failing)
    with pytest.raises(ep.EPError):
        layer.forward(**step())
    refused(layer, calls)
    fails.clear()
    layer.forward(**step())
    layer.backward(GRAD)


def test_refused_arguments_leave_the_last_forward(monkeypatch):
    layer, calls, _ = make(monkeypatch)
    layer.forward(**step())
    calls.clear()
    for bad in (step(x=torch.zeros(N, H)), step(topk_idx=torch.zeros(N, K)), step(topk_weights=torch.zeros(N, K + 1))):
        with pytest.raises(ep.EPError) as err:
            layer.forward(**bad)
        assert err.value.status == ep.EP_ERR_INVALID_ARG
    assert not calls
    layer.backward(GRAD)


def test_before_any_layout_there_are_no_rows(monkeypatch):
    """A forward() that is captured does not run until its graph is replayed; what a backward() before that reads is a layout
    without entries."""
    real = torch.empty

    def dirty(*args, **kw):
        t = real(*args, **kw)
        if t.dim():
            t.view(torch.uint8).fill_(0x55)
        return t

    monkeypatch.setattr(torch, "empty", dirty)
    layer = TrainableExperts(1, N, *weights(), K)
    v = layer.layout.views()
    assert (v["dst_row"] == -1).all() and (v["expert_base"] == 0).all() and (v["recv_cnt"] == 0).all()
    assert (layer.layout.rows_used == 0).all() and (layer._entries() == layer.row_weights.numel() - 1).all()


def test_weights_that_no_product_takes():
    """Refused when the object is made, not halfway through its first forward()."""
    w13, w2 = weights()
    odd = torch.zeros(E, 2 * I + 1, H, dtype=torch.bfloat16)
    for a, b in ((odd, w2), (w13.transpose(1, 2).contiguous().transpose(1, 2), w2), (w13, w2.transpose(1, 2).contiguous().transpose(1, 2)),
                 weights(H=H + 4), (w13[0], w2), (w13.float(), w2.float()), weights(I=I + 8)):
        with pytest.raises(ep.EPError) as err:
            TrainableExperts(1, N, a, b, K)
        assert err.value.status == ep.EP_ERR_INVALID_ARG
