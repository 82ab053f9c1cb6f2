"""Trains a language model's head and decodes with it on 4-bit weights.

    python examples/language_head.py [--steps 60] [--fmt nvfp4|mxfp4]

The hidden states are synthetic: each word has a direction of its own, and a
state is its next word's direction in noise.  Training runs the norm, the
vocabulary cross entropy and both backward passes; decoding freezes the
vocabulary weights in 4 bits and picks the next word of one state at a time.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from precision_transformer_gemms_gb300 import lpq  # noqa: E402
from precision_transformer_gemms_gb300.head import LanguageHead  # noqa: E402


def batch(g, directions, tokens, noise=0.7):
    words = torch.randint(0, directions.shape[0], (tokens,), generator=g, device="cuda")
    x = directions[words] + noise * torch.randn(tokens, directions.shape[1], generator=g, device="cuda")
    labels = torch.where(torch.rand(tokens, generator=g, device="cuda") < 0.1, -100, words)  # some are padding
    return x.bfloat16(), labels, words


def train_and_decode(steps=60, fmt=lpq.NVFP4, d=256, v=1000, tokens=2048, seed=0, say=print):
    """Returns (first loss, last loss, share of words decoded right one by one,
    the same through the prompt's GEMM)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    directions = torch.randn(v, d, generator=g, device="cuda")
    master = {"weight": torch.ones(d, device="cuda"), "bias": torch.zeros(d, device="cuda"),
              "w": 0.02 * torch.randn(v, d, generator=g, device="cuda")}
    rate = {"weight": 0.05, "bias": 0.05, "w": 4.0}
    losses = []
    for step in range(steps):
        head = LanguageHead(master["weight"], master["bias"], master["w"].bfloat16())
        x, labels, _ = batch(g, directions, tokens)
        loss, saved = head.loss(x, labels)
        grads = head.backward(saved)
        for name in master:  # plain gradient descent on fp32 master weights
            master[name].sub_(rate[name] * grads[name].float())
        losses.append(loss)
    losses = torch.stack(losses).tolist()
    say(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {steps} steps")
    head = LanguageHead(master["weight"], master["bias"], master["w"].bfloat16()).freeze(fmt)
    x, _, words = batch(g, directions, 256)
    picked = torch.cat([head.logits(x[i:i + 1]).argmax(1) for i in range(x.shape[0])])
    right = (picked == words).float().mean().item()
    say(f"{lpq.FORMAT_NAMES[fmt]} weights, one token at a time: {100 * right:.1f}% of the next words")
    prompt = (head.prompt_logits(x).argmax(1) == words).float().mean().item()
    say(f"the same states as one prompt (activations in 4 bits too): {100 * prompt:.1f}%")
    return losses[0], losses[-1], right, prompt


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--fmt", choices=("nvfp4", "mxfp4"), default="nvfp4")
    a = p.parse_args()
    train_and_decode(a.steps, lpq.NVFP4 if a.fmt == "nvfp4" else lpq.MXFP4)
