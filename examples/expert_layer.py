"""One expert layer, prefill and decode: residual add and norm, a softmax top-k router in torch,
then the experts (combine_ep_layout_03_gb300.expert_layer).  Random int8 weights.

    python examples/expert_layer.py [--tokens 4096] [--hidden 4096] [--inner 1024] [--experts 128] [--topk 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from combine_ep_layout_03_gb300.expert_layer import ExpertLayer  # noqa: E402


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 4096), ("inner", 1024), ("experts", 128), ("topk", 8)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    H, I, E, K = a.hidden, a.inner, a.experts, a.topk
    g = torch.Generator(device="cuda").manual_seed(0)

    def int8(*shape):
        return torch.empty(shape, dtype=torch.int8, device="cuda").random_(-100, 101, generator=g)

    w13, w2 = int8(E, 2 * I, H), int8(E, H, I)
    s13 = torch.full((E, 2 * I), 0.02 / H ** 0.5, device="cuda")
    s2 = torch.full((E, H), 0.02 / I ** 0.5, device="cuda")
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    gate = torch.randn(H, E, device="cuda", generator=g).to(torch.bfloat16) / H ** 0.5

    for tokens in (a.tokens, 8, 1):   # a prefill chunk, then decoding
        layer = ExpertLayer(1, tokens, w13, s13, w2, s2, gamma, K, alpha=128 if tokens > 64 else 1)
        x = torch.randn(tokens, H, device="cuda", generator=g).to(torch.bfloat16)
        residual = torch.randn(tokens, H, device="cuda", generator=g).to(torch.bfloat16)

        def step():
            y = layer.norm(x, residual)
            weights, idx = (y @ gate).float().softmax(1).topk(K, 1)
            return layer.experts(idx, weights)

        for _ in range(3):
            step()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(10):
            out = step()
        end.record()
        torch.cuda.synchronize()
        print(f"{tokens} tokens ({'few tokens' if layer.few else 'dispatch'}): {start.elapsed_time(end) * 100:.1f} us a step, "
              f"status {layer.status()}, output rms {out.float().square().mean().sqrt().item():.4f}")


if __name__ == "__main__":
    main()
