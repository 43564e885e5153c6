"""One expert layer, prefill and decode: residual add and norm, a softmax top-k router in torch,
then the experts (combine_ep_layout_03_gb300.expert_layer).  Random weights in int8, FP8 or bf16; with --train,
forward and backward of the experts in bf16 instead.

    python examples/expert_layer.py [--tokens 4096] [--hidden 4096] [--inner 1024] [--experts 128] [--topk 8]
                                    [--weights int8|fp8|bf16] [--train]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from combine_ep_layout_03_gb300.expert_layer import ExpertLayer, TrainableExperts  # noqa: E402


def weights_of(kind, E, H, I, g):
    """(w13, its scales, w2, its scales), random."""
    def random(*shape):
        k = shape[-1]
        if kind == "int8":
            w = torch.empty(shape, dtype=torch.int8, device="cuda").random_(-100, 101, generator=g)
            return w, torch.full(shape[:2], 0.02 / k ** 0.5, device="cuda")
        w = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, 100.0 if kind == "fp8" else k ** -0.5, generator=g)
        if kind == "bf16":
            return w, None
        blocks = 2 * ((shape[1] // 2 + 127) // 128) if shape[1] == 2 * I else (shape[1] + 127) // 128
        return w.clamp_(-448, 448).to(torch.float8_e4m3fn), torch.full((E, blocks, k // 128), 0.01 / k ** 0.5, device="cuda")
    return (*random(E, 2 * I, H), *random(E, H, I))


def timed(what, step, status):
    for _ in range(3):
        step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        out = step()
    end.record()
    torch.cuda.synchronize()
    print(f"{what}: {start.elapsed_time(end) * 100:.1f} us a step, status {status()}, output rms "
          f"{out.float().square().mean().sqrt().item():.4f}")


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 4096), ("inner", 1024), ("experts", 128), ("topk", 8)):
        p.add_argument(f"--{name}", type=int, default=value)
    p.add_argument("--weights", choices=("int8", "fp8", "bf16"), default="int8")
    p.add_argument("--train", action="store_true")
    a = p.parse_args()
    H, I, E, K = a.hidden, a.inner, a.experts, a.topk
    g = torch.Generator(device="cuda").manual_seed(0)
    w13, s13, w2, s2 = weights_of("bf16" if a.train else a.weights, E, H, I, g)
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    gate = torch.randn(H, E, device="cuda", generator=g).to(torch.bfloat16) / H ** 0.5

    if a.train:
        experts = TrainableExperts(1, a.tokens, w13, w2, K, alpha=128)
        x, grad = (torch.randn(a.tokens, H, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
        weights, idx = (x @ gate).float().softmax(1).topk(K, 1)

        def step():
            out = experts.forward(x, idx, weights)
            experts.backward(grad)
            return out

        timed(f"{a.tokens} tokens, forward and backward", step, experts.status)
        return

    for tokens in (a.tokens, 8, 1):   # a prefill chunk, then decoding
        layer = ExpertLayer(1, tokens, w13, s13, w2, s2, gamma, K, alpha=128 if tokens > 64 else 1)
        x = torch.randn(tokens, H, device="cuda", generator=g).to(torch.bfloat16)
        residual = torch.randn(tokens, H, device="cuda", generator=g).to(torch.bfloat16)

        def step():
            y = layer.norm(x, residual)
            weights, idx = (y @ gate).float().softmax(1).topk(K, 1)
            return layer.experts(idx, weights)

        timed(f"{tokens} tokens ({'few tokens' if layer.few else 'dispatch'})", step, layer.status)


if __name__ == "__main__":
    main()
