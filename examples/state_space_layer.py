"""A state space layer for serving, from the library's operators: packed prompts, then single tokens.

    python examples/state_space_layer.py [--width 512] [--heads 16] [--layers 2] [--tokens 8]

Each layer normalises the residual stream into 8-bit codes with a scale a token, projects them,
runs the short convolution over x | B | C, the gated selective scan, and an 8-bit norm before the
output projection.  Random weights; the program prefills prompts of several lengths, decodes some
tokens with the states it kept, and prints how far the decoded hidden states are from those that
prefilling the longer sequences gives.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sherman_morrison_inverse_gb300 as vla  # noqa: E402


def project(codes, scale, w):
    """(codes * scale) w^T: e4m3 codes are exact in bfloat16, the scale goes to the result's rows."""
    return (codes.to(torch.bfloat16) @ w.t()).float().mul_(scale[..., None]).to(torch.bfloat16)


class Layer:
    """Weights of one layer and a pool of its states."""

    def __init__(self, width, heads, head, groups, states, taps, slots, gen):
        dev, inner = "cuda", heads * head
        self.heads, self.head, self.groups, self.states = heads, head, groups, states
        self.inner, self.conv = inner, inner + 2 * groups * states
        rand = lambda *s: torch.randn(*s, generator=gen, device=dev)   # noqa: E731
        self.norm_w, self.out_norm_w = torch.ones(width, device=dev), torch.ones(inner, device=dev)
        self.w_in = (rand(inner + self.conv + heads, width) * width ** -0.5).bfloat16()
        self.w_out = (rand(width, inner) * inner ** -0.5).bfloat16()
        self.conv_w, self.conv_b = rand(self.conv, taps) * taps ** -0.5, torch.zeros(self.conv, device=dev)
        self.A, self.D = -torch.linspace(1, 16, heads, device=dev), torch.ones(heads, device=dev)
        self.dt_bias = torch.log(torch.expm1(torch.logspace(-3, -1, heads, device=dev)))
        self.conv_state = torch.zeros(slots, taps - 1, self.conv, dtype=torch.bfloat16, device=dev)
        self.state = torch.zeros(slots, heads, head, states, device=dev)

    def __call__(self, x, residual, slots, offsets=None):
        """x, residual [tokens, width] -> the layer's output; one token a sequence without offsets."""
        codes, scale = vla.rms_norm(x, self.norm_w, residual, out="e4m3")
        z, u, dt = project(codes, scale, self.w_in).split([self.inner, self.conv, self.heads], -1)
        if offsets is None:
            u = vla.short_conv_step(u, self.conv_w, self.conv_b, self.conv_state, slots=slots)
        else:
            u = vla.short_conv(u, self.conv_w, self.conv_b, self.conv_state, offsets=offsets, slots=slots)
        xs, B, C = u.split([self.inner, self.groups * self.states, self.groups * self.states], -1)
        args = (xs.unflatten(-1, (self.heads, self.head)), dt, self.A, B.unflatten(-1, (self.groups, self.states)),
                C.unflatten(-1, (self.groups, self.states)), self.state)
        more = dict(D=self.D, z=z.unflatten(-1, (self.heads, self.head)), dt_bias=self.dt_bias, slots=slots)
        y = vla.ssm_step(*args, **more) if offsets is None else vla.ssm_scan(*args, offsets=offsets, **more)
        codes, scale = vla.rms_norm(y.flatten(1), self.out_norm_w, out="e4m3")
        return project(codes, scale, self.w_out)


def run(layers, x, slots, offsets=None):
    """Hidden states of a stack: each layer's output joins the residual stream at the next norm."""
    residual = torch.zeros(x.shape, device=x.device)
    for layer in layers:
        x = layer(x, residual, slots, offsets)
    return residual + x


def demo(width=512, heads=16, n_layers=2, n_tokens=8, lens=(5, 300, 64, 1)):
    """Largest relative difference between decoding and prefilling the longer sequences."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    S = len(lens)
    slots = torch.randperm(S, generator=gen, device="cuda").to(torch.int32)
    stack = lambda: [Layer(width, heads, 64, 1, 128, 4, S, gen) for _ in range(n_layers)]   # noqa: E731
    state = gen.get_state()
    served = stack()
    gen.set_state(state)
    whole = stack()
    tokens = [torch.randn(n + n_tokens, width, generator=gen, device="cuda").bfloat16() for n in lens]
    offs = lambda ns: torch.tensor([0, *torch.tensor(ns).cumsum(0).tolist()], dtype=torch.int32, device="cuda")   # noqa: E731
    want = run(whole, torch.cat(tokens), slots, offs([n + n_tokens for n in lens])).split([n + n_tokens for n in lens])
    run(served, torch.cat([t[:n] for t, n in zip(tokens, lens)]), slots, offs(list(lens)))
    worst = 0.0
    for i in range(n_tokens):
        got = run(served, torch.stack([t[n + i] for t, n in zip(tokens, lens)]), slots)
        ref = torch.stack([w[n + i] for w, n in zip(want, lens)])
        worst = max(worst, float((got - ref).norm() / ref.norm()))
    return worst


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=8)
    a = ap.parse_args()
    print(f"decoded against prefilled: {demo(a.width, a.heads, a.layers, a.tokens):.3g} relative")
