"""A gated delta rule block with 8-bit projections, served with the library: prompts of
different lengths in one call, then one token at a time from the states they left.

    python examples/gated_delta_block.py [--width 1024] [--batch 4] [--prompt 500] [--tokens 16]

The block (u is the residual stream, [batch, n, width]):
    y, s           = rms_norm(u, quantize)             e4m3 and a scale per token
    qkv, z, b, dt  = linear_e4m3(y, s, w_in)           width → heads' parts
    q, k, v        = causal_conv(qkv)                  depthwise, four taps, silu
    o              = gated_delta(q, k, v, dt, a, b)
    o, s           = rms_norm(o, gate=z, quantize)     per head, times silu(z)
    u              = linear_e4m3(o, s, w_out, residual=u)
``prefill`` runs it over prompts, ``step`` over one token; both read the parts
of the projection's output as slices.  Run as a program it compares the tokens
decoded one by one with the ones a longer prompt gives, and prints times.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import causal_kernelized_linear_gb300 as la  # noqa: E402


def to_e4m3(w):
    """A weight [out, in] as e4m3 and a scale per row, whose largest value becomes 448."""
    scale = w.float().abs().amax(-1).clamp_min(1e-12) / 448.0
    return (w.float() / scale[:, None]).to(torch.float8_e4m3fn), scale


class GatedDeltaBlock:
    """Weights of one block (random, the usual starting rates and steps)."""

    def __init__(self, width, key_heads=4, heads=8, dim=128, taps=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, device=device, generator=g) * shape[-1] ** -0.5

        self.key_heads, self.heads, self.dim = key_heads, heads, dim
        self.keys, self.values = key_heads * dim, heads * dim
        self.mixed = 2 * self.keys + self.values
        self.norm = torch.ones(width, device=device, dtype=torch.bfloat16)
        self.head_norm = torch.ones(dim, device=device, dtype=torch.bfloat16)
        self.w_in, self.s_in = to_e4m3(normal(self.mixed + self.values + 2 * heads, width))
        self.w_conv = normal(self.mixed, taps).bfloat16()
        self.w_out, self.s_out = to_e4m3(normal(width, self.values))
        step0 = torch.exp(torch.rand(heads, device=device, generator=g) * math.log(100.0) + math.log(1e-3))
        self.dt_bias = step0 + torch.log(-torch.expm1(-step0))      # softplus(dt_bias) = step0
        self.a = -1.0 - 15.0 * torch.rand(heads, device=device, generator=g)

    def _project(self, u):
        y, s = la.rms_norm(u, self.norm, quantize=True)
        return la.linear_e4m3(y, s, self.w_in, self.s_in).split(
            [self.mixed, self.values, self.heads, self.heads], -1)

    def _heads(self, x):
        q, k, v = x.split([self.keys, self.keys, self.values], -1)
        return (q.unflatten(-1, (self.key_heads, self.dim)), k.unflatten(-1, (self.key_heads, self.dim)),
                v.unflatten(-1, (self.heads, self.dim)))

    def _finish(self, o, z, u):
        y, s = la.rms_norm(o.flatten(-2), self.head_norm, gate=z, quantize=True)
        return la.linear_e4m3(y, s, self.w_out, self.s_out, residual=u)

    def prefill(self, u, lengths=None, state=None):
        """u [B, n, width] → (u, state); lengths [B] int32: later tokens are padding."""
        conv_state, delta_state = state if state is not None else (None, None)
        x, z, b, dt = self._project(u)
        x, conv_state = la.causal_conv(x, self.w_conv, state=conv_state, lengths=lengths, return_state=True)
        o, delta_state = la.gated_delta(*self._heads(x), dt, self.a, b, dt_bias=self.dt_bias, state=delta_state,
                                        lengths=lengths, return_state=True)
        return self._finish(o, z, u), (conv_state, delta_state)

    def step(self, u, state):
        """u [B, width], the next token → u; the state is updated in place."""
        conv_state, delta_state = state
        x, z, b, dt = self._project(u)
        x = la.causal_conv_step(conv_state, x, self.w_conv)
        o = la.gated_delta_step(delta_state, *self._heads(x), dt, self.a, b, dt_bias=self.dt_bias)
        return self._finish(o, z, u)


def run(width=1024, batch=4, prompt=500, tokens=16, seed=0):
    """Prefills ragged prompts, decodes ``tokens`` inputs one by one, and returns
    the largest difference from prompts that contain them, over their size (the
    two round differently, which e4m3 shows as up to a step of it)."""
    block = GatedDeltaBlock(width, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    u = torch.randn(batch, prompt + tokens, width, device="cuda", generator=g).bfloat16()
    lens = torch.randint(0, prompt + 1, (batch,), device="cuda", generator=g).to(torch.int32)
    lens[0] = prompt
    rows = torch.arange(batch, device="cuda")
    _, state = block.prefill(u[:, :prompt].contiguous(), lengths=lens)
    whole, _ = block.prefill(u, lengths=lens + tokens)
    worst = 0.0
    for t in range(tokens):
        at = lens.long() + t
        got = block.step(u[rows, at], state)
        ref = whole[rows, at]
        worst = max(worst, ((got - ref).float().abs().max() / ref.float().abs().max()).item())
    if la.last_device_status() != 0:
        raise RuntimeError("device status word set")
    return worst


def _time(f, reps):
    f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(reps):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / reps * 1e3


def main():
    ap = argparse.ArgumentParser()
    for name, default in (("width", 1024), ("batch", 4), ("prompt", 500), ("tokens", 16)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    worst = run(a.width, a.batch, a.prompt, a.tokens)
    print(f"decoded tokens against longer prompts: {worst:.2e} of the largest value")
    block = GatedDeltaBlock(a.width)
    u = torch.randn(a.batch, a.prompt, a.width, device="cuda").bfloat16()
    print(f"prompt {a.batch}x{a.prompt}: {_time(lambda: block.prefill(u), 10):.1f} us")
    _, state = block.prefill(u)
    one = u[:, 0].contiguous()
    print(f"token, batch {a.batch}: {_time(lambda: block.step(one, state), 50):.1f} us")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        block.step(one, state)
    print(f"token in a CUDA graph: {_time(graph.replay, 50):.1f} us")


if __name__ == "__main__":
    main()
