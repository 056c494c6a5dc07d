"""Trains the query and output projections of a small attention-like stack in fp8 with head-wise Muon updates.

    python examples/attention_projections_fp8.py [--tokens 1024] [--steps 30]

The student y = (x Wq^T) Wo^T learns a random teacher of the same form from synthetic
tokens: fp8 forward and backward products, weight gradients straight into the fp32
momentum, each head orthogonalised by itself, weights requantised.  Prints the loss.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from matrix_aware_optimizer_amd import BlockLinear  # noqa: E402


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--width", type=int, default=768)
    ap.add_argument("--head-dim", type=int, default=64)
    args = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    d = args.width
    teacher = [randn(d, d) / d ** 0.5 for _ in range(2)]
    # the update's entries have size eta scale / sqrt(d): scale keeps them a fixed part of the weights'
    how = dict(head_dim=args.head_dim, eta=0.05, decay=0.01, scale=0.2 * (d / args.head_dim) ** 0.5)
    layers = [BlockLinear((randn(d, d) / d ** 0.5).to(torch.bfloat16), heads="rows", **how),
              BlockLinear((randn(d, d) / d ** 0.5).to(torch.bfloat16), heads="cols", **how)]
    losses = []
    for step in range(args.steps):
        x = randn(args.tokens, d).to(torch.bfloat16)
        target = (x.float() @ teacher[0].t()) @ teacher[1].t()
        y = layers[1](layers[0](x))
        loss = (y.float() - target).square().mean()
        loss.backward()
        for layer in layers:
            layer.step()
        losses.append(float(loss.detach()))
        if step % 5 == 0 or step == args.steps - 1:
            print(f"step {step:3d}  loss {losses[-1]:.4f}", flush=True)
    # decoding: one token, no gradients
    with torch.no_grad():
        y = layers[1](layers[0](randn(1, d).to(torch.bfloat16)))
    assert torch.isfinite(y).all()
    return losses


if __name__ == "__main__":
    main()
