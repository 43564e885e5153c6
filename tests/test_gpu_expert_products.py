"""The bf16 product of expert rows and its gradients (ep_expert_matmul_bf16, ep_expert_matmul_grad_rows,
ep_expert_matmul_grad_weights) against float64.

Tolerance, from the arithmetic: a product of two bf16 is exact in float32, and each addition of a sum of L terms is off
by at most 2^-23 of the running magnitude (the tensor cores may cut where they add), so a sum by L 2^-23 sum|terms|.  With
swiglu the error of gate and up (dg, du) makes 1.1 dg |u| + (|silu(g)| + 1.1 dg) du + 2^-20 |c| (|silu'| < 1.1; exp,
quotient and products).  An output in bf16 adds 2^-8 of the value for its rounding, one in float32 2^-24, and one that is
added to what was there another 2^-24 of the sum."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def make(counts, N, K, seed=0, spare=3, align=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    base = [0]
    for c in counts:
        base.append(base[-1] + (c + align - 1) // align * align)
    rows = base[-1] + spare
    a = torch.randn(rows, K, device="cuda", generator=g).to(torch.bfloat16)
    dc = torch.randn(rows, N, device="cuda", generator=g).to(torch.bfloat16)
    for e, c in enumerate(counts):
        a[base[e] + c:base[e + 1]], dc[base[e] + c:base[e + 1]] = 0, 0
    # what lies behind the last segment takes no part
    a[base[-1]:], dc[base[-1]:] = float("nan"), float("inf")
    w = (torch.randn(len(counts), N, K, device="cuda", generator=g) / K ** 0.5).to(torch.bfloat16)
    return dict(a=a, dc=dc, w=w, base=base, dense=False, expert_base=torch.tensor(base, dtype=torch.int32, device="cuda"))


def base_of(c):
    return None if c["dense"] else c["expert_base"]


def forward(c, swiglu=False, stream=None, status=None):
    rows, N = c["a"].shape[0], c["w"].shape[1]
    out = torch.full((rows + 1, N // 2 if swiglu else N), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_matmul_bf16(c["a"], c["w"], base_of(c), out[:rows], swiglu=swiglu, status=status, stream=stream)
    torch.cuda.synchronize()
    assert (out[rows:] == 7).all()
    return out[:rows]


def grad_rows(c, stream=None, status=None):
    rows, K = c["a"].shape
    out = torch.full((rows + 1, K), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_matmul_grad_rows(c["dc"], c["w"], base_of(c), out[:rows], status=status, stream=stream)
    torch.cuda.synchronize()
    assert (out[rows:] == 7).all()
    return out[:rows]


def grad_weights(c, dtype=torch.bfloat16, before=None, stream=None, status=None):
    E, N, K = c["w"].shape
    out = torch.full((E + 1, N, K), 7.0, dtype=dtype, device="cuda")
    if before is not None:
        out[:E] = before
    ep.ep_expert_matmul_grad_weights(c["dc"], c["a"], base_of(c), out[:E], accumulate=before is not None, status=status, stream=stream)
    torch.cuda.synchronize()
    assert (out[E:] == 7).all()
    return out[:E]


def within(got, want, tol, what):
    worst = ((got.double() - want).abs() - tol)
    assert not torch.isnan(worst).any() and worst.max().item() <= 0, (what, worst.max().item())


def segments(c):
    base = [0, c["a"].shape[0]] if c["dense"] else c["base"]
    return [(e, slice(base[e], base[e + 1])) for e in range(len(base) - 1) if base[e] < base[e + 1]]


def check_forward(c, swiglu):
    got, K = forward(c, swiglu), c["w"].shape[2]
    for e, r in segments(c):
        a, w = c["a"][r].double(), c["w"][e].double()
        z, dz = a @ w.t(), K * U * (a.abs() @ w.abs().t())
        if swiglu:
            (g, u), (dg, du) = z.chunk(2, 1), dz.chunk(2, 1)
            silu = g * torch.sigmoid(g)
            z = silu * u
            dz = 1.1 * dg * u.abs() + (silu.abs() + 1.1 * dg) * du + 2.0 ** -20 * z.abs()
        within(got[r], z, dz + 2.0 ** -8 * (z.abs() + dz), ("forward", e))
    assert c["dense"] or (got[c["base"][-1]:] == 7).all()
    return got


def check_grad_rows(c):
    got, N = grad_rows(c), c["w"].shape[1]
    for e, r in segments(c):
        d, w = c["dc"][r].double(), c["w"][e].double()
        z, dz = d @ w, N * U * (d.abs() @ w.abs())
        within(got[r], z, dz + 2.0 ** -8 * (z.abs() + dz), ("rows", e))
    assert c["dense"] or (got[c["base"][-1]:] == 7).all()
    return got


def check_grad_weights(c, dtype=torch.bfloat16, before=None):
    got = grad_weights(c, dtype, before)
    want, tol = torch.zeros(got.shape, dtype=torch.float64, device="cuda"), torch.zeros(got.shape, dtype=torch.float64, device="cuda")
    for e, r in segments(c):
        d, a = c["dc"][r].double(), c["a"][r].double()
        want[e] = d.t() @ a
        tol[e] = (r.stop - r.start) * U * (d.abs().t() @ a.abs())
    tol += (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24) * (want.abs() + tol)
    if before is not None:
        want += before.double()
        tol += 2.0 ** -24 * (want.abs() + tol)
    within(got, want, tol, "weights")
    return got


def check_all(c):
    check_forward(c, False)
    check_grad_rows(c)
    check_grad_weights(c)
    check_grad_weights(c, torch.float32)


@pytest.mark.parametrize("M", [1, 2, 7, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 1000])
def test_one_matrix(M):
    c = make([M], 272, 528, seed=M, spare=0)
    c["dense"] = True
    check_all(c)
    check_forward(c, True)


@pytest.mark.parametrize("N", [8, 24, 64, 72, 256, 264, 520])
@pytest.mark.parametrize("K", [8, 56, 64, 128, 136, 1040])
def test_sizes(N, K):
    c = make([37, 300], N, K, seed=N + K)
    check_all(c)
    check_forward(c, True)


@pytest.mark.parametrize("N", [1, 2, 3, 17, 30, 127, 250, 255, 257, 511, 514])
def test_outputs_of_any_width(N):
    c = make([5, 0, 140, 300], N, 96, seed=N)
    check_forward(c, False)
    if N % 2 == 0:
        check_forward(c, True)


@pytest.mark.parametrize("counts,align", [([0, 0, 0], 1), ([1, 0, 2, 0, 3], 1), ([0, 5, 0], 64), ([130, 1, 0, 257, 64, 128], 128),
                                          ([1] * 40, 1), ([700, 0, 900, 0, 1], 64), ([8] * 512, 1), ([16, 48, 80, 33, 15, 95], 1),
                                          ([65] * 100, 1)])
def test_segments(counts, align):
    c = make(counts, 96, 160, align=align, seed=len(counts))
    check_all(c)
    check_forward(c, True)


def test_segments_that_start_late():
    """expert_base[0] > 0: the rows before it belong to nobody."""
    c = make([100, 200], 64, 96)
    c["base"] = [37, 137, 300]
    c["expert_base"].copy_(torch.tensor(c["base"]))
    got = check_forward(c, False)
    assert (got[:37] == 7).all()
    assert (check_grad_rows(c)[:37] == 7).all()
    check_grad_weights(c, torch.float32)


@pytest.mark.parametrize("counts", [[37, 0, 300], [0, 0]])
def test_accumulated_weights(counts):
    c = make(counts, 72, 136, seed=1)
    g = torch.Generator(device="cuda").manual_seed(9)
    before = torch.randn(len(counts), 72, 136, device="cuda", generator=g)
    got = check_grad_weights(c, torch.float32, before)
    for e, n in enumerate(counts):
        assert n or torch.equal(got[e], before[e])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weights_of_no_rows(dtype):
    out = torch.full((2, 16, 24), 7.0, dtype=dtype, device="cuda")
    rows = torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda"), torch.zeros(0, 24, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_matmul_grad_weights(*rows, torch.zeros(3, dtype=torch.int32, device="cuda"), out)
    assert (out == 0).all()


@pytest.mark.parametrize("rows_each", [6, 200])
def test_bad_segments(rows_each):
    """Too many rows, or segments that do not ascend: an error in the status word, and nothing is written."""
    c = make([rows_each] * 4, 64, 64, spare=0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for base, code in (([0, rows_each, 2 * rows_each, 3 * rows_each, 4 * rows_each + 1], ep.EP_ERR_CAPACITY),
                       ([0, 9, 5, 7, 8], ep.EP_ERR_INVALID_ARG), ([-1, 2, 3, 4, 5], ep.EP_ERR_INVALID_ARG),
                       ([-(2 ** 31), 2, 3, 4, 2 ** 31 - 1], ep.EP_ERR_INVALID_ARG)):
        c["expert_base"].copy_(torch.tensor(base, dtype=torch.int64))
        for call in (forward, grad_rows, grad_weights):
            status.zero_()
            assert (call(c, status=status) == 7).all() and status.item() == code
        assert (forward(c, True) == 7).all()


def test_not_finite_values_stay_in_their_segment():
    c = make([40, 21, 200], 96, 128, spare=0)
    refs = forward(c), grad_rows(c), grad_weights(c)
    c["a"][45], c["dc"][45] = float("nan"), float("inf")   # of the second expert's rows
    got = forward(c), grad_rows(c), grad_weights(c)
    for x, ref in zip(got[:2], refs[:2]):
        assert not torch.isfinite(x[45]).any()
        x[45] = ref[45]
        assert torch.equal(x, ref)
    assert not torch.isfinite(got[2][1]).any()
    assert torch.equal(got[2][0], refs[2][0]) and torch.equal(got[2][2], refs[2][2])
    c["w"][1] = float("nan")
    for x, ref in zip((forward(c), grad_rows(c)), refs):
        assert torch.isnan(x[40:61]).all() and torch.equal(x[:40], ref[:40]) and torch.equal(x[61:], ref[61:])


@pytest.mark.parametrize("counts", [[3] * 16, [150] * 16])
def test_repeats_streams_and_graphs(counts):
    c = make(counts, 320, 512)
    calls = lambda **kw: (forward(c, True, **kw), grad_rows(c, **kw), grad_weights(c, torch.float32, **kw))
    refs, st = calls(), torch.cuda.Stream()
    assert all(torch.equal(x, y) for x, y in zip(refs, calls()))
    st.wait_stream(torch.cuda.current_stream())
    assert all(torch.equal(x, y) for x, y in zip(refs, calls(stream=st)))
    outs = [torch.full_like(r, 7) for r in refs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_expert_matmul_bf16(c["a"], c["w"], c["expert_base"], outs[0], swiglu=True)
        ep.ep_expert_matmul_grad_rows(c["dc"], c["w"], c["expert_base"], outs[1])
        ep.ep_expert_matmul_grad_weights(c["dc"], c["a"], c["expert_base"], outs[2])
    other = make(counts, 320, 512, seed=5)
    for name in ("a", "dc", "w"):
        c[name].copy_(other[name])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, calls()))


def test_gradients_against_differences():
    """sum(dc * c) is linear in a and in w, so a difference of any step is its gradient; steps of 1/2 are exact in bf16."""
    c = make([5, 0, 11], 24, 40, seed=2, spare=0)
    da, dw = grad_rows(c), grad_weights(c, torch.float32)

    def loss(a, w):
        return sum((c["dc"][r].double() * (a[r] @ w[e].t())).sum() for e, r in segments(c))

    a, w = c["a"].double(), c["w"].double()
    for i, j in ((0, 0), (4, 39), (5, 7), (15, 21)):
        step = torch.zeros_like(a)
        step[i, j] = 0.5
        diff = (loss(a + step, w) - loss(a - step, w)).item()
        assert abs(da[i, j].item() - diff) <= 2.0 ** -8 * abs(diff) + 1e-5
    for e, n, k in ((0, 0, 0), (0, 23, 39), (2, 5, 6)):
        step = torch.zeros_like(w)
        step[e, n, k] = 0.5
        diff = (loss(a, w + step) - loss(a, w - step)).item()
        assert abs(dw[e, n, k].item() - diff) <= 1e-5 * (1 + abs(diff))


def test_many_tiles():
    """More tiles than CTA pairs, several for each, over uneven segments."""
    g = torch.Generator().manual_seed(4)
    counts = torch.randint(0, 500, (24,), generator=g).tolist()
    check_all(make(counts, 600, 1032, seed=6))


@pytest.mark.parametrize("counts,N,K", [([100], 72, 4104), ([40, 300], 264, 2000), ([33], 2504, 264), ([3001], 72, 136), ([2], 520, 8200),
                                        ([1999, 0, 1, 60, 4000], 264, 72), ([1700, 1555], 40, 520), ([16384], 136, 264)])
def test_long_sums_of_few_tiles(counts, N, K):
    """Sums that several pairs of CTAs share: of k, of n, and of rows; segments that some of them find nothing of."""
    c = make(counts, N, K, seed=N + K)
    check_all(c)
    check_forward(c, True)
    g = torch.Generator(device="cuda").manual_seed(9)
    check_grad_weights(c, torch.float32, torch.randn(len(counts), N, K, device="cuda", generator=g))
    for call in (forward, grad_rows, lambda c: grad_weights(c, torch.float32)):   # the order of parts is fixed
        first = call(c)
        used = torch.isfinite(first)
        assert all(torch.equal(torch.where(used, first, 0), torch.where(used, call(c), 0)) for _ in range(3))


@pytest.mark.parametrize("counts,swiglu", [([5, 9], False), ([5, 9], True), ([150, 200], False), ([150, 200], True), ([600], False)])
def test_outputs_at_odd_addresses(counts, swiglu):
    """An output that lies on two bytes only has the values of one that lies on sixteen."""
    c = make(counts, 264, 96, seed=3)
    rows, width = c["a"].shape[0], 132 if swiglu else 264
    ref, used = forward(c, swiglu), c["base"][-1]
    for shift in (1, 2, 3):
        flat = torch.full((rows * width + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = flat[shift:shift + rows * width].view(rows, width)
        ep.ep_expert_matmul_bf16(c["a"], c["w"], c["expert_base"], out, swiglu=swiglu)
        assert torch.equal(out, ref) and (out[used:] == 7).all() and (flat[:shift] == 7).all() and (flat[shift + rows * width:] == 7).all()


def test_offsets_past_32_bits():
    """More than 2^31 values of rows, of outputs, and of gradients: the last ones are those of the rows alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, N, K = 270000, 8192, 64
    base = torch.tensor([0, 100, rows - 300, rows], dtype=torch.int32, device="cuda")
    a = torch.randn(rows, K, device="cuda", generator=g).to(torch.bfloat16)
    w = (torch.randn(3, N, K, device="cuda", generator=g) / 8).to(torch.bfloat16)
    out = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_matmul_bf16(a, w, base, out)
    last = torch.empty(300, N, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_matmul_bf16(a[-300:], w[2:], None, last)
    assert torch.equal(out[-300:], last)
    z = a[-300:].double() @ w[2].double().t()
    within(last, z, K * U * (a[-300:].double().abs() @ w[2].double().abs().t()) * 2 + 2.0 ** -8 * z.abs(), "last rows")
    da, da_last = torch.empty_like(a), torch.empty(300, K, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_matmul_grad_rows(out, w, base, da)
    ep.ep_expert_matmul_grad_rows(last, w[2:], None, da_last)
    d, m = last.double(), w[2].double()
    for got in (da[-300:], da_last):
        z, dz = d @ m, N * U * (d.abs() @ m.abs())
        within(got, z, dz + 2.0 ** -8 * (z.abs() + dz), "gradient of the last rows")
    dw = torch.empty(3, N, K, dtype=torch.float32, device="cuda")
    ep.ep_expert_matmul_grad_weights(out, a, base, dw)
    within(dw[2], d.t() @ a[-300:].double(), 302 * U * (d.abs().t() @ a[-300:].double().abs()), "gradient of the last matrix")


def test_added_gradients_of_many_tiles():
    c = make([150, 0, 64, 333, 1, 96, 40, 31], 600, 1032, seed=4)
    g = torch.Generator(device="cuda").manual_seed(9)
    check_grad_weights(c, torch.float32, torch.randn(8, 600, 1032, device="cuda", generator=g))


@pytest.mark.parametrize("dtype,accumulate", [(torch.bfloat16, False), (torch.float32, False), (torch.float32, True)])
def test_weight_gradients_at_odd_addresses(dtype, accumulate):
    """A gradient that lies on four bytes only has the values of one that lies on sixteen."""
    c = make([150, 0, 64], 264, 96, seed=5)
    before = torch.randn(3, 264, 96, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) if accumulate else None
    ref = grad_weights(c, dtype, before)
    step = 4 // ref.element_size()
    for shift in (step, 2 * step, 3 * step):
        flat = torch.full((ref.numel() + 4 * step,), 7.0, dtype=dtype, device="cuda")
        out = flat[shift:shift + ref.numel()].view(ref.shape)
        if accumulate:
            out.copy_(before)
        ep.ep_expert_matmul_grad_weights(c["dc"], c["a"], c["expert_base"], out, accumulate=accumulate)
        assert torch.equal(out, ref) and (flat[:shift] == 7).all() and (flat[shift + ref.numel():] == 7).all()
