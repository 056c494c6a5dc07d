"""Trains a gated feed-forward block with Muon and answers from its int8 codes.

    python examples/gated_block_int8.py [--tokens 1024] [--steps 30]

The student h = act(x Wg^T) * (x Wu^T) learns a random teacher of the same form from
synthetic tokens: bf16 products, weight gradients straight into the fp32 momenta, each
matrix orthogonalised by itself.  Then both weights are quantised to int8 and the block
answers for a prompt and for single tokens.  Prints the loss and the answers' distance.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from matrix_aware_optimizer_amd import GatedLinear  # noqa: E402


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--width", type=int, default=768)
    ap.add_argument("--hidden", type=int, default=2304)
    args = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    d, f = args.width, args.hidden
    teacher = GatedLinear(*((randn(f, d) / d ** 0.5).to(torch.bfloat16) for _ in range(2)))
    block = GatedLinear(*((randn(f, d) / d ** 0.5).to(torch.bfloat16) for _ in range(2)), eta=0.02)
    losses = []
    for step in range(args.steps):
        x = randn(args.tokens, d).to(torch.bfloat16)
        with torch.no_grad():
            target = teacher(x).float()
        loss = (block(x).float() - target).square().mean()
        loss.backward()
        block.step()
        losses.append(float(loss.detach()))
        if step % 5 == 0 or step == args.steps - 1:
            print(f"step {step:3d}  loss {losses[-1]:.4f}", flush=True)
    block.quantize()
    x = randn(100, d).to(torch.bfloat16)
    with torch.no_grad():
        full = block(x).float()
    prompt = block.answer(x).float()
    tokens = torch.cat([block.answer(x[i:i + 1]) for i in range(3)]).float()
    gap = float((prompt - full).norm() / full.norm())
    assert torch.equal(tokens, prompt[:3])       # integer sums are exact: a token alone gets the prompt's answer
    print(f"int8 answers differ from bf16 by {gap:.4f}", flush=True)
    return losses, gap


if __name__ == "__main__":
    main()
