"""The 8-bit integer product of expert rows (ep_expert_matmul) against float64.

Tolerance, from the arithmetic: products of codes are exact in float32 and so are sums up
to 2^24; past that an addition is off by at most 2^-23 of the running magnitude, so a sum of
k terms by k 2^-23 sum|terms| (0 where sum|terms| < 2^24).  Two scales round twice.  With
swiglu the error of gate and up (dg, du) makes 1.1 dg |u| + (|silu(g)| + 1.1 dg) du + 2^-20 |c|
(|silu'| < 1.1; exp, quotient and products).  The output's own rounding adds 2^-8."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def make(counts, N, K, swiglu, align=1, seed=0, full=False, spare=3):
    """Segments of `counts` rows, each padded to a multiple of `align`; `spare` rows past the last."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    E = len(counts)
    aligned = [(c + align - 1) // align * align for c in counts]
    base = [0]
    for c in aligned:
        base.append(base[-1] + c)
    rows = base[-1] + spare
    top = 128 if full else 100
    a = torch.randint(-top, top, (rows, K), device="cuda", generator=g, dtype=torch.int8)
    w = torch.randint(-top, top, (E, N, K), device="cuda", generator=g, dtype=torch.int8)
    if full:
        a[: rows // 2], w[:, ::2] = -128, -128       # the largest sums, beyond 2^24 for long k
    sa = torch.rand(rows, device="cuda", generator=g) * 0.02 + 0.01
    sw = (torch.rand(E, N, device="cuda", generator=g) * 0.02 + 0.01) / K ** 0.5
    for e, c in enumerate(counts):
        a[base[e] + c:base[e + 1]], sa[base[e] + c:base[e + 1]] = 0, 0
    return dict(a=a, a_scales=sa, w=w, w_scales=sw, base=base, swiglu=swiglu, dense=False,
                expert_base=torch.tensor(base, dtype=torch.int32, device="cuda"))


def call(c, stream=None, status=None):
    rows, N = c["a"].shape[0], c["w"].shape[1]
    out = torch.full((rows + 1, N // 2 if c["swiglu"] else N), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_matmul(c["a"], c["a_scales"], c["w"], c["w_scales"], None if c["dense"] else c["expert_base"],
                        out[:rows], swiglu=c["swiglu"], status=status, stream=stream)
    torch.cuda.synchronize()
    assert (out[rows:] == 7).all()
    return out[:rows]


def check(c):
    got = call(c).double()
    base = [0, c["a"].shape[0]] if c["dense"] else c["base"]
    assert (got[base[-1]:] == 7).all(), "rows past the last segment were written"
    K, N = c["w"].shape[2], c["w"].shape[1]
    for e in range(len(base) - 1):
        r = slice(base[e], base[e + 1])
        if r.start == r.stop:
            continue
        a, w = c["a"][r].double(), c["w"][e].double()
        sums, mags = a @ w.t(), a.abs() @ w.abs().t()
        s = c["a_scales"][r].double()[:, None] * c["w_scales"][e].double()
        z = sums * s
        dz = torch.where(mags < 2 ** 24, 0.0, K * U * mags) * s + 4 * U * z.abs()
        if c["swiglu"]:
            (g, u), (dg, du) = z.chunk(2, 1), dz.chunk(2, 1)
            silu = g * torch.sigmoid(g)
            z = silu * u
            dz = 1.1 * dg * u.abs() + (silu.abs() + 1.1 * dg) * du + 2.0 ** -20 * z.abs()
        tol = dz + 2.0 ** -8 * (z.abs() + dz)
        worst = ((got[r] - z).abs() - tol).max().item()
        assert worst <= 0, (e, worst)
    return got


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 127, 128, 129, 256, 257, 300, 1000])
def test_one_matrix(swiglu, M):
    c = make([M], 272, 528, swiglu, seed=M, spare=0)
    c["dense"] = True
    check(c)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N", [2, 6, 16, 30, 250, 256, 258, 514, 1000])
@pytest.mark.parametrize("K", [16, 48, 64, 80, 1040])
def test_sizes(swiglu, N, K):
    check(make([37, 300], N, K, swiglu, seed=N + K))


@pytest.mark.parametrize("N", [1, 3, 17, 127, 255, 257, 511])
def test_odd_outputs(N):
    check(make([5, 0, 140], N, 96, False, seed=N))


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,align", [([0, 0, 0], 1), ([1, 0, 2, 0, 3], 1), ([0, 5, 0], 64), ([130, 1, 0, 257, 64, 128], 128),
                                          ([1] * 40, 1), ([700, 0, 900, 0, 1], 64), ([8] * 512, 1)])
def test_segments(swiglu, counts, align):
    check(make(counts, 96, 160, swiglu, align=align, seed=len(counts)))


@pytest.mark.parametrize("M", [8, 300])
@pytest.mark.parametrize("K", [1024, 4096])
def test_largest_codes(M, K):
    check(make([M], 130, K, False, seed=K, full=True))


@pytest.mark.parametrize("rows_each", [6, 200])
def test_too_few_rows(rows_each):
    c = make([rows_each] * 4, 64, 64, False, spare=0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(c, status=status)
    assert status.item() == ep.EP_OK
    c["expert_base"][-1] += 1
    assert (call(c, status=status) == 7).all() and status.item() == ep.EP_ERR_CAPACITY


@pytest.mark.parametrize("base", [[0, -5, 50, 100], [90, 20, 60, 100], [-(2 ** 31), 10, 2, 100]])
def test_bad_bases_stay_inside(base):
    """Not ascending, or negative: any result, but only inside the buffers."""
    c = make([30, 30, 40], 64, 64, False, spare=0)
    c["expert_base"].copy_(torch.tensor(base, dtype=torch.int32))
    call(c)


@pytest.mark.parametrize("counts", [[3] * 16, [150] * 16])
def test_repeats_streams_and_graphs(counts):
    c = make(counts, 320, 512, True, align=8)
    ref = call(c)
    assert torch.equal(ref, call(c))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    assert torch.equal(ref, call(c, stream=st))
    out = torch.full_like(ref, 7)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_expert_matmul(c["a"], c["a_scales"], c["w"], c["w_scales"], c["expert_base"], out, swiglu=True)
    c["a"].copy_(make(counts, 320, 512, True, align=8, seed=5)["a"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, call(c))


def test_not_finite_scales_stay_in_their_row():
    c = make([40, 200], 96, 128, False, spare=0)
    ref = call(c)
    c["a_scales"][50] = float("nan")
    got = call(c)
    assert torch.isnan(got[50]).all()
    got[50] = ref[50]
    assert torch.equal(got, ref)


def test_receive_rows_of_a_layout():
    """The rows and segments of a dispatch, as they are."""
    R, T, H, E, K = 2, 50, 256, 8, 2
    lay = ep.EPLayout(R, T, H, E, K, 16)
    g = torch.Generator(device="cuda").manual_seed(3)
    idx = torch.rand(R * T, E, device="cuda", generator=g).topk(K, 1).indices.view(R, T, K)
    lay.layout(idx)
    x = torch.randn(R * T, H, device="cuda", generator=g).to(torch.bfloat16)
    data, scales = lay.alloc_recv(ep.EP_QUANT_INT8_PER_TOKEN)
    lay.dispatch(x, ep.EP_QUANT_INT8_PER_TOKEN, data, scales)
    w = torch.randint(-90, 90, (E, 64, H), device="cuda", generator=g, dtype=torch.int8)
    sw = torch.rand(E, 64, device="cuda", generator=g) / 1000
    out = torch.zeros(data.shape[0], 64, dtype=torch.bfloat16, device="cuda")
    lay.expert_matmul(data, scales, w, sw, out)
    assert lay.status() == ep.EP_OK
    base = lay.views()["expert_base"].tolist()
    for e in range(E):
        r = slice(base[e], base[e + 1])
        want = (data[r].view(torch.int8).double() @ w[e].double().t()) * scales[r].view(torch.float32).double() * sw[e].double()
        assert ((out[r].double() - want).abs() <= 2.0 ** -7 * want.abs()).all()
    y = torch.zeros(data.shape[0], 32, dtype=torch.bfloat16, device="cuda")
    lay.expert_matmul(data[: base[-1] - 1], scales[: base[-1] - 1], w, sw, y[: base[-1] - 1], swiglu=True)
    assert lay.status() == ep.EP_ERR_CAPACITY and (y == 0).all()
