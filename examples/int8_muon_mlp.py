"""Trains a small network kept only in bf16: its matrices' products run in 8-bit
integers (forward and backward), and its matrices are updated by Muon, its
vectors by AdamW, both written back by stochastic rounding.  Then serves it one
token at a time from weights quantised once.

    python examples/int8_muon_mlp.py [--steps N] [--width W] [--tokens T]

Synthetic data: a fixed random network of the same shape is the target.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from stochastic_rounding_gb300 import (AdamWSR, Int8Linear, MuonSR, asr_quantize_int8, int8_empty,  # noqa: E402
                                       int8_linear)


class Network(torch.nn.Module):
    def __init__(self, width, seed):
        super().__init__()
        self.up = Int8Linear(width, 4 * width, seed=seed, device="cuda")
        self.down = Int8Linear(4 * width, width, seed=seed + 1, device="cuda")
        self.bias = torch.nn.Parameter(torch.zeros(width, dtype=torch.bfloat16, device="cuda"))

    def forward(self, x):
        return x + self.down(torch.relu(self.up(x))) + self.bias


def train(steps=60, width=256, tokens=512, seed=0):
    """Returns the losses and the network."""
    torch.manual_seed(seed)
    target, net = Network(width, 100), Network(width, 7)
    muon = MuonSR([net.up.weight, net.down.weight], lr=0.02, weight_decay=0.01, seed=1)
    adamw = AdamWSR([net.bias], lr=1e-2, weight_decay=0.0, seed=2)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, device="cuda").to(torch.bfloat16)
        with torch.no_grad():
            want = target(x).float()
        loss = (net(x).float() - want).square().mean()
        muon.zero_grad(), adamw.zero_grad()
        loss.backward()
        muon.step(), adamw.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist(), net


def serve(net, tokens):
    """The network's outputs for one token after another, from weights quantised once."""
    quantised = []
    for layer in (net.up, net.down):
        w = layer.weight.detach()
        quantised.append(asr_quantize_int8(w, int8_empty(*w.shape), torch.empty(w.shape[0], device="cuda")))
    out = []
    for x in tokens.split(1):
        h = torch.relu(int8_linear(x, *quantised[0]))
        out.append(x + int8_linear(h, *quantised[1]) + net.bias.detach())
    return torch.cat(out)


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    a.add_argument("--steps", type=int, default=60)
    a.add_argument("--width", type=int, default=256)
    a.add_argument("--tokens", type=int, default=512)
    a = a.parse_args()
    losses, net = train(a.steps, a.width, a.tokens)
    print(f"loss: first {losses[0]:.4f}, last {losses[-1]:.4f}")
    x = torch.randn(8, a.width, device="cuda").to(torch.bfloat16)
    with torch.no_grad():
        print("served tokens equal the batch's:", torch.equal(serve(net, x), net(x)))
