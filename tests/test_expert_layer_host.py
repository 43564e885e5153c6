"""What ExpertLayer hands to the library, on the CPU: its tensors are CPU tensors here, and the
library's calls are replaced by ones that keep what they are given."""
import contextlib
import ctypes
import random

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from combine_ep_layout_03_gb300 import ep
from combine_ep_layout_03_gb300.expert_layer import STATUS_WORDS, ExpertLayer

E, H, I, K = 4, 64, 16, 2


def make(R, T, few, monkeypatch):
    """A layer of either way, and the list of (call, its tensors) that experts() fills."""
    f = torch.zeros
    layer = ExpertLayer(R, T, f(E, 2 * I, H, dtype=torch.int8), f(E, 2 * I), f(E, H, I, dtype=torch.int8), f(E, H),
                        f(H, dtype=torch.bfloat16), K, few_tokens=64 if few else 0)
    assert layer.few == few
    calls = []

    def keep(name):
        def call(*args, **kw):
            calls.append((name, args, kw))
        return call

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(ep, "ep_moe_few_tokens", keep("few"))
    monkeypatch.setattr(ep, "ep_quant_rows", keep("quant_rows"))
    if not few:
        for name in ("layout", "dispatch_ex", "expert_matmul", "combine"):
            monkeypatch.setattr(layer.layout, name, keep(name))
    return layer, calls


def routing(N):
    return torch.zeros(N, K, dtype=torch.int64), torch.zeros(N, K)


def shared_of(calls, few):
    """The shared rows that the kernels were given, as [R, S, T, H] or [S, N, H]."""
    name, args, kw = calls[-1]
    assert name == ("few" if few else "combine")
    return args[9] if few else args[3]


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("R,T,S", [(1, 8, 1), (1, 8, 3), (2, 4, 1), (2, 4, 3), (4, 1, 2)])
@pytest.mark.parametrize("by_rank", [False, True])
def test_shared_rows_reach_the_kernels_in_their_order(few, R, T, S, by_rank, monkeypatch):
    """combine reads R x S x T rows, the few-token kernels S x N: both get as many as they read, each
    token its own, whichever of the two documented shapes the caller has."""
    layer, calls = make(R, T, few, monkeypatch)
    ranks = torch.randn(R, S, T, H).to(torch.bfloat16)
    tokens = ranks.transpose(0, 1).reshape(S, R * T, H)
    layer.experts(*routing(R * T), ranks if by_rank else tokens)
    got = shared_of(calls, few)
    assert got.is_contiguous() and torch.equal(got, tokens if few else ranks)


@pytest.mark.parametrize("few", [False, True])
def test_shared_rows_of_other_shapes_are_refused(few, monkeypatch):
    layer, calls = make(2, 4, few, monkeypatch)
    bf = torch.bfloat16
    for shape in ((8, H), (3, 4, H), (3, 8, H + 8), (1, 3, 8, H), (2, 3, 8, H), (2, 4, 3, H), (2, 3, 4, H // 2), (1, 2, 3, 4, H)):
        with pytest.raises(ep.EPError) as err:
            layer.experts(*routing(8), torch.zeros(shape, dtype=bf))
        assert err.value.status == ep.EP_ERR_INVALID_ARG
    with pytest.raises(ep.EPError):
        layer.experts(*routing(8), torch.zeros(2, 3, 4, H))
    assert not calls or calls[-1][0] not in ("few", "combine")


@pytest.mark.parametrize("few", [False, True])
def test_routing_of_other_types_and_sizes_is_refused(few, monkeypatch):
    """bf16 router weights, say, would be read as float32 past their end."""
    layer, calls = make(2, 4, few, monkeypatch)
    idx, wts = routing(8)
    for a, b in ((idx.int(), wts), (idx[:4], wts), (idx.t().contiguous().t(), wts), (torch.cat([idx, idx]), wts),
                 (idx, wts.to(torch.bfloat16)), (idx, wts.double()), (idx, wts[:4]), (idx, wts[:, :1]),
                 (idx, wts.t().contiguous().t()), (idx, torch.zeros(8, 2 * K)[:, ::2])):
        with pytest.raises(ep.EPError) as err:
            layer.experts(a, b)
        assert err.value.status == ep.EP_ERR_INVALID_ARG
    assert not calls
    for a, b in ((idx, wts), (idx.view(2, 4, K), wts.view(2, 4, K))):
        layer.experts(a, b)


class Streams:
    """Stands in for torch's streams: `now` is the one that an operation would run on."""

    def __init__(self, monkeypatch):
        self.now = "current"
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("handle", handle))
        monkeypatch.setattr(torch.cuda, "stream", self.enter)

    @contextlib.contextmanager
    def enter(self, stream):
        before, self.now = self.now, stream
        yield
        self.now = before

    @contextlib.contextmanager
    def writes(self):
        """The list of (operation that writes a tensor, its stream) of what runs inside."""
        seen, streams = [], self

        class Record(TorchDispatchMode):
            def __torch_dispatch__(self, func, types, args=(), kwargs=None):
                if func.overloadpacket in (torch.ops.aten.clone, torch.ops.aten.copy_, torch.ops.aten._to_copy, torch.ops.aten.zero_,
                                           torch.ops.aten._local_scalar_dense):
                    seen.append((func.overloadpacket, streams.now))
                return func(*args, **(kwargs or {}))

        with Record():
            yield seen


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("stream,runs_on", [(None, "current"), ("side", "side"), (1 << 40, ("handle", 1 << 40))])
def test_shared_rows_are_reordered_on_the_calls_stream(few, stream, runs_on, monkeypatch):
    """A copy on another stream than the kernels' may not be there yet when they read it."""
    layer, calls = make(2, 4, few, monkeypatch)
    streams = Streams(monkeypatch)
    shared = torch.randn(3, 8, H).to(torch.bfloat16) if not few else torch.randn(2, 3, 4, H).to(torch.bfloat16)
    with streams.writes() as seen:
        layer.experts(*routing(8), shared, stream=stream)
    copies = [s for op, s in seen if op in (torch.ops.aten.clone, torch.ops.aten.copy_)]
    assert copies and set(copies) == {runs_on}


def erring(monkeypatch):
    """A list whose first entry the next steps of the few-token way leave in their status words."""
    error = [ep.EP_OK]

    def few_tokens(*args):
        word = ctypes.c_int32.from_address(args[10])
        if word.value == 0:   # the kernels keep the first error
            word.value = error[0]

    monkeypatch.setattr(ep, "ep_moe_few_tokens", few_tokens)
    return error


def test_status_is_that_of_the_last_step(monkeypatch):
    """Bad ids, good steps, other errors, over more steps than there are status words: each step's own."""
    layer, _ = make(1, 8, True, monkeypatch)
    streams, error, rng, clears = Streams(monkeypatch), erring(monkeypatch), random.Random(0), []
    for step in range(2 * STATUS_WORDS + 100):
        stream = rng.choice([None, "side"])
        error[0] = rng.choice([ep.EP_OK, ep.EP_OK, ep.EP_ERR_BAD_EXPERT_ID, ep.EP_ERR_TIMEOUT])
        with streams.writes() as seen:
            layer.experts(*routing(8), stream=stream)
        clears += [(step, on == (stream or "current")) for op, on in seen if op is torch.ops.aten.zero_]
        with streams.writes() as seen:
            assert layer.status(stream) == error[0]
        assert seen == [(torch.ops.aten._local_scalar_dense, stream or "current")]
    assert len(clears) == 2 and all(on_the_steps_stream for _, on_the_steps_stream in clears)


def test_replays_of_captured_steps_report_each_error_once(monkeypatch):
    layer, _ = make(1, 8, True, monkeypatch)
    streams, error, replay = Streams(monkeypatch), erring(monkeypatch), []
    bad = error[0] = ep.EP_ERR_BAD_EXPERT_ID
    layer.experts(*routing(8))
    assert layer.status() == bad
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(ep, "ep_moe_few_tokens", lambda *args, keep=ep.ep_moe_few_tokens: replay.append(lambda: keep(*args)))
    with streams.writes() as seen:
        layer.experts(*routing(8), stream="side")
    assert not seen   # nothing but the layer's kernels in the graph
    for errors, want in (((ep.EP_OK,), ep.EP_OK), ((bad,), bad), ((ep.EP_OK,), ep.EP_OK), ((bad, ep.EP_OK), bad),
                         ((ep.EP_ERR_TIMEOUT, bad), ep.EP_ERR_TIMEOUT), ((ep.EP_OK,), ep.EP_OK)):
        for error[0] in errors:
            replay[0]()
        with streams.writes() as seen:
            assert layer.status("side") == want
        assert all(on == "side" for _, on in seen)


@pytest.mark.parametrize("R,T,S", [(1, 0, 2), (2, 0, 2), (2, 4, 0)])
def test_no_tokens_or_no_shared_rows(R, T, S, monkeypatch):
    layer, calls = make(R, T, True, monkeypatch)
    for shared in (torch.zeros(R, S, T, H, dtype=torch.bfloat16), torch.zeros(S, R * T, H, dtype=torch.bfloat16)):
        layer.experts(*routing(R * T), shared)
        assert shared_of(calls, True).shape == (S, R * T, H)
