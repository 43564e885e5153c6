"""Kernels that are set up while the one before them ends still see all that it wrote: chains in which each call reads what the
one before has just written, eagerly and as a graph, have the values of the same calls with a synchronisation after each."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

pytestmark = pytest.mark.gpu


def bf16(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def products(E, M, H, I):
    """c = x w13^T, inner and its codes, y = inner w2^T; back through all of it; weights' gradients added; x from y and dx."""
    rows, f32 = E * M, torch.float32
    base = torch.arange(E + 1, dtype=torch.int32, device="cuda") * M
    x, w13, w2 = bf16(rows, H, seed=1), bf16(E, 2 * I, H, seed=2, scale=H ** -0.5), bf16(E, H, I, seed=3, scale=I ** -0.5)
    c, inner, codes = torch.empty_like(bf16(rows, 2 * I, seed=4)), bf16(rows, I, seed=5), torch.empty(rows, 2 * I, dtype=torch.uint8, device="cuda")
    scales, dinner, dc = torch.empty(rows, 2 * I // 128, device="cuda"), bf16(rows, I, seed=6), bf16(rows, 2 * I, seed=7)
    y, dx = bf16(rows, H, seed=8), bf16(rows, H, seed=9)
    dw13, dw2 = torch.zeros(E, 2 * I, H, device="cuda", dtype=f32), torch.zeros(E, H, I, device="cuda", dtype=f32)
    calls = [lambda: ep.ep_expert_matmul_bf16(x, w13, base, c),
             lambda: ep.ep_swiglu_keep(c, inner, codes, scales),
             lambda: ep.ep_expert_matmul_bf16(inner, w2, base, y),
             lambda: ep.ep_expert_matmul_grad_rows(y, w2, base, dinner),
             lambda: ep.ep_expert_matmul_grad_weights(y, inner, base, dw2, accumulate=True),
             lambda: ep.ep_swiglu_keep_grad(codes, scales, dinner, dc, inner=inner),
             lambda: ep.ep_expert_matmul_grad_weights(dc, x, base, dw13, accumulate=True),
             lambda: ep.ep_expert_matmul_grad_rows(dc, w13, base, dx),
             lambda: ep.ep_expert_matmul_bf16(dx, w13, base, c, swiglu=False),
             lambda: ep.ep_expert_matmul_bf16(dx, w13, base, x.view(-1)[:rows * I].view(rows, I), swiglu=True)]
    return calls, (x, c, inner, codes, scales, y, dinner, dc, dx, dw13, dw2)


def eight_bits(E, M, H):
    """FP8 and int8 products and quantisations in turn, each of what the one before wrote."""
    rows = E * M
    base = torch.arange(E + 1, dtype=torch.int32, device="cuda") * M
    g = torch.Generator(device="cuda").manual_seed(1)
    w8 = (torch.randn(E, H, H, device="cuda", generator=g) * 16).to(torch.float8_e4m3fn)
    s8 = torch.full((E, (H + 127) // 128, H // 128), 1 / 16 / H ** 0.5, device="cuda")
    wi, si = torch.randint(-127, 128, (E, H, H), device="cuda", dtype=torch.int8, generator=g), torch.full((E, H), 1 / 73 / H ** 0.5, device="cuda")
    x = bf16(rows, H, seed=3)
    fp8, fs = torch.empty(rows, H, dtype=torch.uint8, device="cuda"), torch.empty(rows, H // 128, device="cuda")
    i8, i8s = torch.empty(rows, H, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    calls = [lambda: ep.ep_quant_rows(x, ep.EP_QUANT_FP8_E4M3_PER_GROUP, fp8, fs),
             lambda: ep.ep_expert_matmul_fp8(fp8, fs, w8, s8, base, x),
             lambda: ep.ep_quant_rows(x, ep.EP_QUANT_INT8_PER_TOKEN, i8, i8s),
             lambda: ep.ep_expert_matmul(i8, i8s, wi, si, base, x)]
    return calls, (x, fp8, fs, i8, i8s)


@pytest.mark.parametrize("make,sizes", [(products, (1, 3, 128, 128)), (products, (4, 40, 256, 128)), (products, (16, 150, 512, 384)),
                                        (products, (2, 700, 1024, 256)), (eight_bits, (1, 4, 256)), (eight_bits, (4, 50, 512)),
                                        (eight_bits, (16, 200, 1024))])
def test_chains(make, sizes):
    turns = 4
    calls, state = make(*sizes)
    start = [t.clone() for t in state]

    def reset():
        for t, s in zip(state, start):
            t.copy_(s)
        torch.cuda.synchronize()

    for _ in range(turns):
        for call in calls:
            call()
            torch.cuda.synchronize()
    want = [t.clone() for t in state]
    assert not torch.equal(want[0], start[0])

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(t.view(torch.uint8), w.view(torch.uint8)) for t, w in zip(state, want))

    for _ in range(5):
        reset()
        for _ in range(turns):
            for call in calls:
                call()
        assert same()
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in calls:
            call()
    for _ in range(5):
        reset()
        for _ in range(turns):
            graph.replay()
        assert same()
