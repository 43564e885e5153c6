"""The FP8 product of expert rows with a scale for each block of 128 (ep_expert_matmul_fp8) against float64.

Tolerance, from the arithmetic: a product of two e4m3 is exact in float32, and each addition of a block's 128 terms is off
by at most 2^-23 of the running magnitude (the tensor cores may cut where they add); the two scales' product, its product
with the sum and the addition of each of B blocks are off by 2^-24 each.  So a sum by (128 + B + 2) 2^-23 of its terms'
magnitudes.  With swiglu the error of gate and up (dg, du) makes 1.1 dg |u| + (|silu(g)| + 1.1 dg) du + 2^-20 |c| (|silu'| <
1.1; exp, quotient and products).  The output's rounding adds 2^-8."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def codes_of(g, *shape):
    v = torch.randn(*shape, device="cuda", generator=g) * 100
    return v.clamp_(-448, 448).to(torch.float8_e4m3fn)


def make(counts, N, K, swiglu, seed=0, spare=3, align=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    base = [0]
    for c in counts:
        base.append(base[-1] + (c + align - 1) // align * align)
    rows, E = base[-1] + spare, len(counts)
    halves = 2 if swiglu else 1
    a, w = codes_of(g, rows, K), codes_of(g, E, N, K)
    sa = torch.rand(rows, K // 128, device="cuda", generator=g) * 0.02 + 0.001
    sw = (torch.rand(E, halves * ((N // halves + 127) // 128), K // 128, device="cuda", generator=g) * 0.02 + 0.001) / K ** 0.5
    for e, c in enumerate(counts):
        a[base[e] + c:base[e + 1]], sa[base[e] + c:base[e + 1]] = 0, 0
    a[base[-1]:], sa[base[-1]:] = float("nan"), float("inf")   # what lies behind the last segment takes no part
    return dict(a=a, sa=sa, w=w, sw=sw, base=base, swiglu=swiglu, dense=False,
                expert_base=torch.tensor(base, dtype=torch.int32, device="cuda"))


def call(c, stream=None, status=None):
    rows, N = c["a"].shape[0], c["w"].shape[1]
    out = torch.full((rows + 1, N // 2 if c["swiglu"] else N), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_matmul_fp8(c["a"], c["sa"], c["w"], c["sw"], None if c["dense"] else c["expert_base"], out[:rows],
                            swiglu=c["swiglu"], status=status, stream=stream)
    torch.cuda.synchronize()
    assert (out[rows:] == 7).all()
    return out[:rows]


def matrix(c, e):
    """Expert e's weights and scales, one for each value."""
    N, K = c["w"].shape[1:]
    halves = c["sw"][e].double().chunk(2 if c["swiglu"] else 1)
    size = N // len(halves)
    return c["w"][e].double() * torch.cat([h.repeat_interleave(128, 0)[:size] for h in halves]).repeat_interleave(128, 1)


def check(c):
    got = call(c)
    base = [0, c["a"].shape[0]] if c["dense"] else c["base"]
    blocks = c["w"].shape[2] // 128
    for e in range(len(base) - 1):
        r = slice(base[e], base[e + 1])
        if r.start == r.stop:
            continue
        a, w = c["a"][r].double() * c["sa"][r].double().repeat_interleave(128, 1), matrix(c, e)
        z, dz = a @ w.t(), (128 + blocks + 2) * U * (a.abs() @ w.abs().t())
        if c["swiglu"]:
            (g, u), (dg, du) = z.chunk(2, 1), dz.chunk(2, 1)
            silu = g * torch.sigmoid(g)
            z = silu * u
            dz = 1.1 * dg * u.abs() + (silu.abs() + 1.1 * dg) * du + 2.0 ** -20 * z.abs()
        worst = (got[r].double() - z).abs() - (dz + 2.0 ** -8 * (z.abs() + dz))
        assert not torch.isnan(worst).any() and worst.max().item() <= 0, (e, worst.max().item())
    assert c["dense"] or (got[base[-1]:] == 7).all()
    return got


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 300, 1000])
def test_one_matrix(swiglu, M):
    c = make([M], 272, 512, swiglu, seed=M, spare=0)
    c["dense"] = True
    check(c)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N", [2, 6, 16, 30, 32, 64, 126, 128, 250, 256, 258, 512, 514, 1000])
@pytest.mark.parametrize("counts", [[20, 30], [37, 150], [37, 500]])
def test_widths(swiglu, N, counts):
    check(make(counts, N, 256, swiglu, seed=N))


@pytest.mark.parametrize("N", [1, 3, 17, 127, 255, 257, 511])
@pytest.mark.parametrize("M", [5, 140, 500])
def test_odd_outputs(N, M):
    check(make([M, 0, 5], N, 128, False, seed=N))


@pytest.mark.parametrize("K", [128, 256, 384, 640, 1280, 4096])
@pytest.mark.parametrize("M", [9, 100, 420])
def test_lengths(K, M):
    check(make([M, 2 * M], 96, K, False, seed=K + M))
    check(make([M, 2 * M], 192, K, True, seed=K + M))


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,align", [([0, 0, 0], 1), ([1, 0, 2, 0, 3], 1), ([0, 5, 0], 64), ([130, 1, 0, 257, 64, 128], 128),
                                          ([1] * 40, 1), ([700, 0, 900, 0, 1], 64), ([8] * 512, 1), ([65] * 100, 1), ([300] * 40, 1)])
def test_segments(swiglu, counts, align):
    check(make(counts, 320, 256, swiglu, align=align, seed=len(counts)))


@pytest.mark.parametrize("rows_each", [6, 100, 300])
def test_bad_segments(rows_each):
    """Too many rows, or segments that do not ascend: an error in the status word, and nothing is written."""
    c = make([rows_each] * 4, 64, 128, False, spare=0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(c, status=status)
    assert status.item() == ep.EP_OK
    for base, code in (([0, rows_each, 2 * rows_each, 3 * rows_each, 4 * rows_each + 1], ep.EP_ERR_CAPACITY),
                       ([0, 9, 5, 7, 8], ep.EP_ERR_INVALID_ARG), ([-1, 2, 3, 4, 5], ep.EP_ERR_INVALID_ARG)):
        c["expert_base"].copy_(torch.tensor(base))
        status.zero_()
        assert (call(c, status=status) == 7).all() and status.item() == code


@pytest.mark.parametrize("M", [10, 100, 300])
def test_largest_codes(M):
    c = make([M], 130, 2048, False, seed=M)
    c["a"].fill_(448)
    c["w"].fill_(-448)
    check(c)


@pytest.mark.parametrize("counts", [[10, 20], [100, 90], [300, 250]])
def test_not_finite_values_stay_where_they_enter(counts):
    c = make(counts, 320, 256, False, spare=0)
    ref, r = call(c), counts[0] + 4
    c["sa"][r, 1] = float("nan")
    got = call(c)
    assert torch.isnan(got[r]).all()
    got[r] = ref[r]
    assert torch.equal(got, ref)
    c = make(counts, 320, 256, False, spare=0)
    c["a"][r, 7] = float("nan")
    c["sw"][1, 2, 0] = float("nan")      # channels 256 to 319 of the second expert
    got = call(c)
    assert torch.isnan(got[r]).all() and torch.isnan(got[counts[0]:, 256:]).all()
    got[r], got[counts[0]:, 256:] = ref[r], ref[counts[0]:, 256:]
    assert torch.equal(got, ref)


@pytest.mark.parametrize("counts", [[3] * 16, [70] * 16, [250] * 16])
def test_repeats_streams_and_graphs(counts):
    c = make(counts, 320, 512, True)
    ref, st = call(c), torch.cuda.Stream()
    assert torch.equal(ref, call(c))
    st.wait_stream(torch.cuda.current_stream())
    assert torch.equal(ref, call(c, stream=st))
    out = torch.full_like(ref, 7)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_expert_matmul_fp8(c["a"], c["sa"], c["w"], c["sw"], c["expert_base"], out, swiglu=True)
    c["a"].copy_(make(counts, 320, 512, True, seed=5)["a"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, call(c))


def test_receive_rows_of_a_layout():
    """The rows, scales and segments of a dispatch, as they are."""
    R, T, H, E, K = 2, 50, 256, 8, 2
    lay = ep.EPLayout(R, T, H, E, K, 16)
    g = torch.Generator(device="cuda").manual_seed(3)
    lay.layout(torch.rand(R * T, E, device="cuda", generator=g).topk(K, 1).indices.view(R, T, K))
    x = torch.randn(R * T, H, device="cuda", generator=g).to(torch.bfloat16)
    data, scales = lay.alloc_recv(ep.EP_QUANT_FP8_E4M3_PER_GROUP)
    lay.dispatch(x, ep.EP_QUANT_FP8_E4M3_PER_GROUP, data, scales)
    c = make([1] * E, 130, H, False)
    base = lay.views()["expert_base"]
    c.update(a=data, sa=scales, expert_base=base)
    got = call(c)
    c.update(a=data.view(torch.float8_e4m3fn), sa=scales.view(torch.float32), base=base.tolist())
    assert torch.equal(got, check(c))


@pytest.mark.parametrize("counts", [[5, 9], [60, 20], [300, 500]])
@pytest.mark.parametrize("swiglu", [False, True])
def test_outputs_at_odd_addresses(counts, swiglu):
    """An output that lies on two bytes only has the values of one that lies on sixteen."""
    c = make(counts, 272, 256, swiglu, seed=3)
    rows, width = c["a"].shape[0], 136 if swiglu else 272
    ref = call(c)
    for shift in (1, 4):
        flat = torch.full((rows * width + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = flat[shift:shift + rows * width].view(rows, width)
        ep.ep_expert_matmul_fp8(c["a"], c["sa"], c["w"], c["sw"], c["expert_base"], out, swiglu=swiglu)
        assert torch.equal(out, ref) and (flat[:shift] == 7).all() and (flat[shift + rows * width:] == 7).all()


def test_offsets_past_32_bits():
    """More than 2^31 codes of rows and outputs: the last ones are those of the rows alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, N, K = 530000, 4096, 4224
    a = torch.empty(rows, K, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    a.view(torch.uint8).zero_()
    sa = torch.zeros(rows, K // 128, device="cuda")
    a[-300:], sa[-300:] = codes_of(g, 300, K), torch.rand(300, K // 128, device="cuda", generator=g)
    w, sw = codes_of(g, 2, N, K), torch.rand(2, N // 128, K // 128, device="cuda", generator=g)
    base = torch.tensor([0, rows - 300, rows], dtype=torch.int32, device="cuda")
    out = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_matmul_fp8(a, sa, w, sw, base, out)
    assert (out[rows // 2] == 0).all()
    c = dict(a=a[-300:], sa=sa[-300:], w=w[1:], sw=sw[1:], base=[0, 300], swiglu=False, dense=True)
    alone = check(c)
    assert torch.equal(out[-300:], alone)
