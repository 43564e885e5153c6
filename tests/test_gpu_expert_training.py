"""The expert layer with FP8 and bf16 weights, and its experts in training (ExpertLayer, TrainableExperts): each step against
float64 of what that step was given, and the whole against the formula.

Steps round once to bf16 (2^-8 of the value) and a sum of L terms is off by L 2^-23 of its terms' magnitudes (FP8: a block of
128 and then the blocks, fewer than L); the 2-norms of the whole are derived where they are used."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep
from combine_ep_layout_03_gb300.expert_layer import ExpertLayer, TrainableExperts

pytestmark = pytest.mark.gpu

BF16, U = 2.0 ** -8, 2.0 ** -23
SHAPES = [(1, 200, 512, 8, 2, 256, 1), (2, 300, 1024, 16, 4, 384, 128), (4, 33, 256, 64, 8, 128, 16)]


def within(got, want, tol, what=""):
    worst = (got.double() - want).abs() - tol
    assert not torch.isnan(worst).any() and worst.max().item() <= 0, (what, worst.max().item())


def routing(g, N, E, K, drop=0.1):
    idx = torch.rand(N, E, device="cuda", generator=g).topk(K, 1).indices
    idx[torch.rand(N, K, device="cuda", generator=g) < drop] = -1
    return idx, torch.softmax(torch.randn(N, K, device="cuda", generator=g), 1)


def product(a, w):
    """a w^T and the bound of its float32 sum."""
    return a @ w.t(), a.shape[1] * U * (a.abs() @ w.abs().t())


def blocks(codes, scales, halves=1):
    """Codes times a scale for each 128 x 128 (each half's rows counted apart)."""
    size = codes.shape[0] // halves
    rows = torch.cat([h.repeat_interleave(128, 0)[:size] for h in scales.double().chunk(halves)])
    return codes.double() * rows.repeat_interleave(128, 1)


def quantised(g, E, n, k, halves):
    w = torch.randn(E, n, k, device="cuda", generator=g) / k ** 0.5
    size = n // halves
    codes, scales = torch.empty(E, n, k, device="cuda"), []
    for e in range(E):
        parts = []
        for h in range(halves):
            part = torch.nn.functional.pad(w[e, h * size:(h + 1) * size], (0, 0, 0, -size % 128)).view(-1, 128, k // 128, 128)
            s = part.abs().amax((1, 3)) / 448
            codes[e, h * size:(h + 1) * size] = (part / s[:, None, :, None]).view(-1, k)[:size]
            parts.append(s)
        scales.append(torch.cat(parts))
    return codes.clamp(-448, 448).to(torch.float8_e4m3fn), torch.stack(scales)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("R,T,H,E,K,I,alpha", SHAPES)
def test_layer(fp8, R, T, H, E, K, I, alpha):
    g = torch.Generator(device="cuda").manual_seed(E)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    if fp8:
        (w13, s13), (w2, s2) = quantised(g, E, 2 * I, H, 2), quantised(g, E, H, I, 1)
    else:
        w13, s13 = (r(E, 2 * I, H) / H ** 0.5).to(torch.bfloat16), None
        w2, s2 = (r(E, H, I) / I ** 0.5).to(torch.bfloat16), None
    layer = ExpertLayer(R, T, w13, s13, w2, s2, (1 + 0.1 * r(H)).to(torch.bfloat16), K, alpha=alpha)
    idx, wts = routing(g, R * T, E, K)
    y = layer.norm(r(R * T, H).to(torch.bfloat16), r(R * T, H).to(torch.bfloat16))
    shared = r(R, 2, T, H).to(torch.bfloat16)
    out = layer.experts(idx, wts, shared)
    assert layer.status() == ep.EP_OK and not layer.few
    v = layer.layout.views()
    dst, base = v["dst_row"].view(-1, K).long(), v["expert_base"].tolist()
    hit = dst >= 0
    token = torch.arange(R * T, device="cuda")[:, None].expand(-1, K)[hit]
    if fp8:
        assert torch.equal(layer.recv[dst[hit]], layer.rows.view(torch.uint8)[token])
        recv = layer.recv.view(torch.float8_e4m3fn).double() * layer.recv_scales.view(torch.float32).double().repeat_interleave(128, 1)
        inner = layer.inner_rows.double() * layer.inner_scales.double().repeat_interleave(128, 1)
    else:
        assert torch.equal(layer.recv[dst[hit]], y[token])
        recv, inner = layer.recv.double(), layer.inner.double()
    want_out = shared.double().sum(1).reshape(R * T, H)
    whole = want_out.clone()
    for e in range(E):
        s = slice(base[e], base[e + 1])
        a = blocks(w13[e], s13[e], 2) if fp8 else w13[e].double()
        b = blocks(w2[e], s2[e]) if fp8 else w2[e].double()
        z, dz = product(recv[s], a)
        (gate, up), (dg, du) = z.chunk(2, 1), dz.chunk(2, 1)
        silu = gate * torch.sigmoid(gate)
        want = silu * up
        tol = 1.1 * dg * up.abs() + (silu.abs() + 1.1 * dg) * du + 2.0 ** -20 * want.abs()
        within(layer.inner[s], want, tol + BF16 * (want.abs() + tol), "inner")
        want, tol = product(inner[s], b)
        within(layer.expert_out[s], want, tol + BF16 * (want.abs() + tol), "out of experts")
        here = (idx == e).any(1).nonzero()[:, 0]
        gate, up = (y[here].double() @ a.t()).chunk(2, 1)
        whole[here] += torch.where(idx == e, wts, 0.0).sum(1)[here].double()[:, None] * ((gate * torch.sigmoid(gate) * up) @ b.t())
    terms = torch.where(hit[:, :, None], layer.expert_out[dst.clamp_min(0)].double() * wts.double()[:, :, None], 0.0)
    terms = torch.cat([terms, shared.double().transpose(0, 1).reshape(2, R * T, H).transpose(0, 1)], 1)
    within(out, terms.sum(1), BF16 * terms.sum(1).abs() + (2 * K + 5) * 2.0 ** -24 * terms.abs().sum(1), "combine")
    # the whole, against unquantised activations: bf16 rounds inner rows, experts' rows and the result (2^-8 each; inner's
    # passes through a linear product).  FP8 adds two quantisations of rows, a code off by at most 2^-4 of it, evenly
    # spread: below 2^-4 / sqrt(3) = 0.037 of a row's norm each, the first at most doubled by SwiGLU's two factors.
    assert (out.double() - whole).norm() <= (0.12 if fp8 else 3 * BF16) * whole.norm()


@pytest.mark.parametrize("T", [1, 40])
def test_few_tokens_with_bf16_weights(T):
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    w13, w2 = (r(8, 256, 256) / 16).to(torch.bfloat16), (r(8, 256, 128) / 11).to(torch.bfloat16)
    gamma, x = torch.ones(256, device="cuda", dtype=torch.bfloat16), r(T, 256).to(torch.bfloat16)
    few, more = (ExpertLayer(1, T, w13, None, w2, None, gamma, 2, few_tokens=n) for n in (64, 0))
    assert few.few and not more.few
    idx, wts = routing(g, T, 8, 2, 0.0)
    few.norm(x), more.norm(x)
    a, b = few.experts(idx, wts).double(), more.experts(idx, wts).double()
    assert few.status() == more.status() == ep.EP_OK
    assert (a - b).norm() <= 4 * BF16 * a.norm()   # one way rounds inner rows and experts' rows, both the result


class Step:
    def __init__(self, R, T, H, E, K, I, alpha, seed=0, drop=0.1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.w13, self.w2 = (r(E, 2 * I, H) / H ** 0.5).to(torch.bfloat16), (r(E, H, I) / I ** 0.5).to(torch.bfloat16)
        self.layer = TrainableExperts(R, T, self.w13, self.w2, K, alpha)
        self.x, self.grad = r(R * T, H).to(torch.bfloat16), r(R * T, H).to(torch.bfloat16)
        self.idx, self.wts = routing(g, R * T, E, K, drop)

    def run(self, stream=None):
        out = self.layer.forward(self.x, self.idx, self.wts, stream)
        return (out, *self.layer.backward(self.grad, stream))


@pytest.mark.parametrize("R,T,H,E,K,I,alpha", SHAPES)
def test_training_step(R, T, H, E, K, I, alpha):
    s = Step(R, T, H, E, K, I, alpha, seed=E)
    layer = s.layer
    out = layer.forward(s.x, s.idx, s.wts)
    c, inner, expert_out = layer.c.double(), layer.inner.double(), layer.expert_out.double()
    grad_x, grad_wts = layer.backward(s.grad)
    assert layer.status() == ep.EP_OK
    v = layer.layout.views()
    dst, base = v["dst_row"].view(-1, K).long(), v["expert_base"].tolist()
    hit, used = dst >= 0, base[-1]
    token = torch.arange(R * T, device="cuda")[:, None].expand(-1, K)[hit]
    weights = torch.zeros(used, dtype=torch.float64, device="cuda")
    weights[dst[hit]] = s.wts[hit].double()
    assert torch.equal(layer.row_weights[:used].double(), weights)
    assert torch.equal(layer.rows[dst[hit]], s.x[token]) and torch.equal(layer.expert_out[dst[hit]], s.grad[token])
    kept = layer.codes.double() * layer.scales.double().repeat_interleave(128, 1)
    w = weights[:, None]
    for e in range(E):
        r = slice(base[e], base[e + 1])
        rows, d = layer.rows[r].double(), layer.expert_out[r].double()
        within(c[r], *[z for z in (lambda z, dz: (z, dz + BF16 * (z.abs() + dz)))(*product(rows, s.w13[e].double()))], "c")
        gate, up = c[r].chunk(2, 1)
        want = w[r] * gate * torch.sigmoid(gate) * up
        within(inner[r], want, (BF16 + 2.0 ** -15) * want.abs() + 1e-30, "inner")   # (|g| + 8) 2^-22 below 2^-15
        z, dz = product(inner[r], s.w2[e].double())
        within(expert_out[r], z, dz + BF16 * (z.abs() + dz), "out of experts")
        # backward, from what was kept
        dy, tol = product(d, s.w2[e].double().t())
        within(layer.grad_inner[r], dy, tol + BF16 * (dy.abs() + tol), "gradient of inner rows")
        dy, (gate, up) = layer.grad_inner[r].double(), kept[r].chunk(2, 1)
        sig = torch.sigmoid(gate)
        want = torch.cat([w[r] * dy * up * (sig + gate * sig * (1 - sig)), w[r] * dy * gate * sig], 1)
        scale = torch.cat([(w[r] * dy * up).abs() * (1 + gate.abs()), want[:, I:].abs()], 1)
        within(layer.c[r], want, BF16 * want.abs() + 2.0 ** -15 * scale + 1e-30, "gradient of c")
        terms = dy * gate * sig * up
        within(layer.row_weights_grad[r], terms.sum(1), (I * U + 2.0 ** -15) * terms.abs().sum(1) + 1e-30, "gradient of weights")
        again = w[r] * gate * sig * up
        within(layer.inner[r], again, (BF16 + 2.0 ** -15) * again.abs() + 1e-30, "inner again")
        for got, left, right in ((layer.grad_w2[e], d, layer.inner[r].double()), (layer.grad_w13[e], layer.c[r].double(), rows)):
            n = r.stop - r.start
            within(got, left.t() @ right, (n + 2) * U * (left.abs().t() @ right.abs()), "gradient of matrices")
        dx, tol = product(layer.c[r].double(), s.w13[e].double().t())
        within(layer.grad_rows[r], dx, tol + BF16 * (dx.abs() + tol), "gradient of rows")
    for got, rows in ((out, expert_out), (grad_x, layer.grad_rows.double())):
        terms = torch.where(hit[:, :, None], rows[dst.clamp_min(0)], 0.0)
        within(got, terms.sum(1), BF16 * terms.sum(1).abs() + (K + 1) * 2.0 ** -24 * terms.abs().sum(1), "sum of a token")
    assert torch.equal(grad_wts[hit], layer.row_weights_grad[dst[hit]]) and (grad_wts[~hit] == 0).all()


def formula(s, x, wts, w13, w2):
    out = torch.zeros(s.layer.N, s.layer.H, dtype=torch.float64, device="cuda")
    for e in range(s.layer.E):
        weight = torch.where(s.idx == e, wts, torch.zeros((), dtype=torch.float64, device="cuda")).sum(1)
        gate, up = (x @ w13[e].t()).chunk(2, 1)
        out = out + weight[:, None] * ((gate * torch.sigmoid(gate) * up) @ w2[e].t())
    return out


def test_gradients_are_those_of_the_formula():
    """Against automatic differentiation of the layer's formula in float64.  Kept gates and ups are off by at most 2^-4 of
    themselves, evenly spread: 0.037 of a row's norm.  A gradient has one or two such factors (a gate's through the
    slope of silu, which changes less than twice as fast as the gate), so 0.12 bounds the relative 2-norm."""
    s = Step(2, 96, 256, 8, 2, 256, 8, seed=5)
    leaves = [t.double().requires_grad_() for t in (s.x, s.wts, s.w13, s.w2)]
    want = formula(s, *leaves)
    want.backward(s.grad.double())
    out, grad_x, grad_wts = s.run()
    assert (out.double() - want).norm() <= 4 * BF16 * want.norm()
    for got, leaf in zip((grad_x, grad_wts, s.layer.grad_w13, s.layer.grad_w2), leaves):
        assert (got.double() - leaf.grad).norm() <= 0.12 * leaf.grad.norm()


def test_steps_add_up_and_leave_nothing_behind():
    """Gradients of weights add up over steps; a step's other results do not depend on the one before."""
    s = Step(1, 150, 256, 16, 4, 128, 64, seed=6)
    first = s.run()
    w13, w2 = s.layer.grad_w13.clone(), s.layer.grad_w2.clone()
    other = Step(1, 150, 256, 16, 4, 128, 64, seed=7)
    s.layer.zero_grad()
    assert (s.layer.grad_w13 == 0).all()
    x, idx, wts = s.x, s.idx, s.wts
    s.x, s.idx, s.wts = other.x * 100, other.idx, torch.full_like(other.wts, float("nan"))   # a bad step between
    s.run()
    s.x, s.idx, s.wts = x, idx, wts
    s.layer.zero_grad()
    again = s.run()
    assert all(torch.equal(a, b) for a, b in zip(first, again)) and torch.equal(s.layer.grad_w13, w13) and torch.equal(s.layer.grad_w2, w2)
    s.run()
    assert torch.equal(s.layer.grad_w13, w13 + w13) and torch.equal(s.layer.grad_w2, w2 + w2)


def test_router_weights_of_a_graph_of_their_own():
    """Weights that require gradients (a softmax over the router's output) leave no graph behind in the layer."""
    s = Step(1, 60, 256, 8, 2, 128, 1, seed=3)
    ref = s.run()
    logits = torch.log(s.wts).requires_grad_()
    s.wts = torch.softmax(logits, 1)
    for _ in range(2):
        out, grad_x, grad_wts = s.run()
        assert not (out.requires_grad or grad_x.requires_grad or grad_wts.requires_grad or s.layer.row_weights.requires_grad)
    s.wts.backward(grad_wts)
    assert torch.isfinite(logits.grad).all() and (out - ref[0]).double().norm() <= 4 * BF16 * ref[0].double().norm()


def test_no_entry_has_an_expert():
    s = Step(1, 20, 256, 4, 2, 128, 1, drop=2.0)
    out, grad_x, grad_wts = s.run()
    assert (out == 0).all() and (grad_x == 0).all() and (grad_wts == 0).all() and (s.layer.grad_w2 == 0).all()


def test_on_another_stream_and_captured():
    s = Step(1, 150, 256, 16, 4, 128, 1, seed=8)
    ref = s.run()
    w13 = s.layer.grad_w13.clone()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    s.layer.zero_grad(st)
    got = s.run(st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got)) and torch.equal(s.layer.grad_w13, w13)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.layer.zero_grad()
        outs = s.run()
    other = Step(1, 150, 256, 16, 4, 128, 1, seed=9)
    for name in ("x", "idx", "wts", "grad", "w13", "w2"):
        getattr(s, name).copy_(getattr(other, name))
    graph.replay()
    torch.cuda.synchronize()
    want = other.run()
    assert all(torch.equal(a, b) for a, b in zip(want, outs)) and torch.equal(s.layer.grad_w13, other.layer.grad_w13)


def test_refusals():
    s = Step(1, 20, 256, 4, 2, 128, 1)
    for a in ((s.x.float(), s.idx, s.wts), (s.x[:10], s.idx, s.wts), (s.x, s.idx.int(), s.wts), (s.x, s.idx, s.wts.double()),
              (s.x, s.idx, s.wts[:, :1]), (s.x.t().contiguous().t(), s.idx, s.wts)):
        with pytest.raises(ep.EPError) as err:
            s.layer.forward(*a)
        assert err.value.status == ep.EP_ERR_INVALID_ARG
    for bad in (s.grad.float(), s.grad[:10], s.grad.t().contiguous().t()):
        with pytest.raises(ep.EPError):
            s.layer.backward(bad)
    for w13, w2 in ((s.w13.float(), s.w2), (s.w13, s.w2[:, :, :64]), (s.w13[:, :192].contiguous(), s.w2[:, :, :96].contiguous())):
        with pytest.raises(ep.EPError):
            TrainableExperts(1, 20, w13, w2, 2)
