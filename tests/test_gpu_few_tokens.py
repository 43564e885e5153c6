"""The expert layer of a few tokens (ep_moe_few_tokens) against float64.

Tolerance, from the arithmetic: a product of bf16 (or int8) values is exact in float32,
and a float32 sum of n terms in any order, each addition off by at most 2^-23 of the
running magnitude (the tensor cores may truncate), is off by n 2^-23 sum|terms|.  With
dg and du the bounds of gate and up (two more roundings where scales multiply them), the
inner value h = w silu(g) u is off by
    dh = |w| (1.1 dg |u| + (|silu(g)| + 1.1 dg) du) + 2^-19 |h|        (|silu'| < 1.1)
(exp, quotient and products within 2^-20, the bf16 pair within 2^-18 / 2), and the output
by sum|W2| dh + (n I + 9 + S) 2^-23 (sum|W2 h| + sum|shared|) and its own rounding, 2^-8."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def make(T, H, E, K, I, int8, S=0, seed=0, drop=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x = r(T, H).to(torch.bfloat16)
    idx = torch.rand(T, E, device="cuda", generator=g).topk(K, 1).indices if T else torch.zeros(0, K, dtype=torch.int64, device="cuda")
    idx[torch.rand(T, K, device="cuda", generator=g) < drop] = -1
    wts = torch.softmax(r(T, K), 1) if T else torch.zeros(0, K, device="cuda")
    if int8:
        w13 = (r(E, 2 * I, H) * 40).round().clamp(-128, 127).to(torch.int8)
        w2 = (r(E, H, I) * 40).round().clamp(-128, 127).to(torch.int8)
        s13 = (torch.rand(E, 2 * I, device="cuda", generator=g) + 0.5) / 40 / H ** 0.5
        s2 = (torch.rand(E, H, device="cuda", generator=g) + 0.5) / 40 / I ** 0.5
    else:
        w13, w2 = (r(E, 2 * I, H) / H ** 0.5).to(torch.bfloat16), (r(E, H, I) / I ** 0.5).to(torch.bfloat16)
        s13 = s2 = None
    shared = r(S, T, H).to(torch.bfloat16) if S else None
    return dict(x=x, topk_idx=idx, topk_weights=wts, w13=w13, w2=w2, w13_scales=s13, w2_scales=s2, shared=shared)


def call(c, stream=None, status=None):
    T, H = c["x"].shape
    E, I, K = c["w13"].shape[0], c["w13"].shape[1] // 2, c["topk_idx"].shape[1]
    n = ep.ep_moe_few_tokens_workspace_size(T, H, E, K, I)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")    # NaN patterns: what is not written shows
    out = torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_moe_few_tokens(c["x"], c["topk_idx"], c["topk_weights"], c["w13"], c["w2"], out[:T], ws[:n],
                         w13_scales=c["w13_scales"], w2_scales=c["w2_scales"], shared=c["shared"], stream=stream,
                         status=status)
    torch.cuda.synchronize()
    assert (out[T:] == 7).all() and (ws[n:] == 0xFF).all()
    return out[:T]


def reference(c):
    """(value, error bound) in float64."""
    x, idx, wts = c["x"].double(), c["topk_idx"], c["topk_weights"].double()
    T, H = x.shape
    E, I = c["w13"].shape[0], c["w13"].shape[1] // 2
    S = 0 if c["shared"] is None else c["shared"].shape[0]
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    mag, err = out.clone(), out.clone()
    n = torch.zeros(T, 1, dtype=torch.float64, device="cuda")
    for e in sorted(set(idx.flatten().tolist())):
        if not 0 <= e < E:
            continue
        hit = idx == e
        w = torch.where(hit, wts, 0.0).sum(1)
        t = hit.any(1).nonzero()[:, 0]
        w13, w2 = c["w13"][e].double(), c["w2"][e].double()
        if c["w13_scales"] is not None:
            w13, w2 = w13 * c["w13_scales"][e].double()[:, None], w2 * c["w2_scales"][e].double()[:, None]
        z, dz = x[t] @ w13.t(), (H + 10) * U * (x[t].abs() @ w13.abs().t())
        (g, u), (dg, du) = z.chunk(2, 1), dz.chunk(2, 1)
        silu, a = g * torch.sigmoid(g), w[t][:, None]
        h = a * silu * u
        dh = a.abs() * (1.1 * dg * u.abs() + (silu.abs() + 1.1 * dg) * du) + 2.0 ** -19 * h.abs()
        out[t] += h @ w2.t()
        mag[t] += h.abs() @ w2.abs().t()
        err[t] += dh @ w2.abs().t()
        n[t] += 1
    if S:
        out += c["shared"].double().sum(0)
        mag += c["shared"].double().abs().sum(0)
    err += (n * I + 9 + S) * U * mag
    return out, err + 2.0 ** -8 * (out.abs() + err)


def check(c, got=None):
    got = (call(c) if got is None else got).double()
    want, tol = reference(c)
    worst = ((got - want).abs() - tol).max().item() if got.numel() else 0
    assert worst <= 0, worst
    return got


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T,H,E,K,I", [(1, 1024, 16, 2, 512), (1, 16, 1, 1, 16), (2, 48, 3, 3, 16), (5, 1024, 16, 2, 352),
                                       (8, 528, 8, 4, 80), (9, 256, 4, 2, 64), (16, 1040, 8, 8, 144), (17, 512, 2, 2, 48),
                                       (40, 512, 64, 8, 96), (64, 1024, 512, 16, 32), (64, 256, 4, 1, 272)])
def test_sizes(int8, T, H, E, K, I):
    check(make(T, H, E, K, I, int8, seed=T + H))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T,H,E,K,I", [(8, 272, 64, 8, 1232), (20, 272, 64, 8, 1232), (8, 1600, 64, 8, 208),
                                       (16, 2192, 32, 8, 176), (50, 144, 128, 4, 656), (5, 2480, 16, 4, 1104)])
def test_work_split_over_warps_and_ctas(int8, T, H, E, K, I):
    """Tiles shared by two, four or eight warps, the last group short; output tiles of two and three CTAs."""
    check(make(T, H, E, K, I, int8, seed=T + I, drop=0.1))


@pytest.mark.parametrize("T,H,I", [(3, 8, 8), (7, 24, 40), (33, 1000, 104)])
def test_odd_bf16_sizes(T, H, I):
    check(make(T, H, 6, 3, I, False, S=1, seed=I))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("S", [1, 4])
def test_shared_rows_and_dropped_entries(int8, S):
    c = make(13, 512, 16, 4, 128, int8, S=S, drop=0.5, seed=4)
    c["topk_idx"][3] = -1                      # a token without an expert: its shared rows alone
    got = check(c)
    want = c["shared"].float().sum(0)[3].to(torch.bfloat16).double()
    assert torch.equal(got[3], want)


@pytest.mark.parametrize("T", [1, 8, 64])
def test_no_entry_at_all(T):
    c = make(T, 256, 8, 2, 64, False, seed=T)
    c["topk_idx"][:] = -1
    c["topk_weights"][:] = float("nan")        # weights of absent entries are not read into the sum
    assert (call(c) == 0).all()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T", [8, 16, 31, 64])
def test_all_tokens_on_one_expert(int8, T):
    c = make(T, 512, 8, 2, 128, int8, seed=T)
    c["topk_idx"][:, 0], c["topk_idx"][:, 1] = 5, -1
    check(c)


def test_an_expert_named_twice():
    c = make(6, 256, 8, 4, 64, False, seed=2)
    c["topk_idx"][:, 2] = c["topk_idx"][:, 0]
    check(c)


def test_bad_ids_are_absent_and_reported():
    c = make(4, 256, 8, 2, 64, False, seed=3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(c, status=status)
    assert status.item() == ep.EP_OK
    d = dict(c, topk_idx=c["topk_idx"].clone())
    d["topk_idx"][1, 0], d["topk_idx"][2, 1] = 8, -2
    got = call(d, status=status)
    assert status.item() == ep.EP_ERR_BAD_EXPERT_ID
    d["topk_idx"][1, 0] = d["topk_idx"][2, 1] = -1
    assert torch.equal(got, call(d))


def test_a_nan_stays_with_its_token():
    c = make(20, 256, 4, 2, 64, False, seed=6)
    ref = call(c)
    c["x"][11, 3] = float("nan")
    got = call(c)
    keep = [t for t in range(20) if t != 11]
    assert torch.equal(got[keep], ref[keep]) and torch.isnan(got[11]).all()


@pytest.mark.parametrize("int8", [False, True])
def test_repeats_streams_and_graphs(int8):
    c = make(24, 1024, 32, 4, 256, int8, S=1, drop=0.1, seed=7)
    ref = call(c)
    assert torch.equal(ref, call(c))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    assert torch.equal(ref, call(c, stream=st))
    out = torch.empty_like(ref)
    ws = torch.empty(24 * 4 * 256 * 4, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_moe_few_tokens(c["x"], c["topk_idx"], c["topk_weights"], c["w13"], c["w2"], out, ws,
                             w13_scales=c["w13_scales"], w2_scales=c["w2_scales"], shared=c["shared"])
    other = make(24, 1024, 32, 4, 256, int8, S=1, drop=0.1, seed=8)
    for k in ("x", "topk_idx", "topk_weights", "shared"):
        c[k].copy_(other[k])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, call(c))


def test_int8_weights_are_their_scaled_values():
    """The largest codes, both signs, and -128."""
    c = make(3, 128, 2, 1, 32, True, seed=9)
    c["w13"][:] = torch.tensor([-128, 127, -127, 1, -1, 0, 64, -64], dtype=torch.int8, device="cuda").repeat(16)
    check(c)
