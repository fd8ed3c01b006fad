"""A selective state-space block served with the library: prompts of different
lengths in one call, then one token at a time from the states they left.

    python examples/state_space_block.py [--width 1024] [--batch 4] [--prompt 500] [--tokens 16]

The block (u is the residual stream, [batch, n, width]):
    x, gate   = linear(rmsnorm(u), w_in)               width → 2·inner
    x         = causal_conv(x)                         depthwise, four taps, silu
    dt, b, c  = linear(x, w_x)                         inner → rank + 2·states
    dt        = linear(dt, w_dt)                       rank → inner
    y         = selective_scan(x, dt, a, b, c, skip, gate)
    u         = linear(y, w_out, residual=u)
``prefill`` runs it over prompts, ``step`` over one token; both read the parts
of a projection's output as slices.  Run as a program it checks that the
tokens decoded one by one are the ones a longer prompt gives, and prints times.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import causal_kernelized_linear_gb300 as la  # noqa: E402


class StateSpaceBlock:
    """Weights of one block (random, the usual starting rates and steps)."""

    def __init__(self, width, states=16, taps=4, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        inner, rank = 2 * width, max(8, width // 16 // 8 * 8)

        def normal(*shape):
            return (torch.randn(*shape, device=device, generator=g) * shape[-1] ** -0.5).to(dtype)

        self.width, self.inner, self.rank, self.states, self.taps = width, inner, rank, states, taps
        self.norm = torch.ones(width, device=device, dtype=dtype)
        self.w_in = normal(2 * inner, width)
        self.w_conv, self.b_conv = normal(inner, taps), torch.zeros(inner, device=device, dtype=dtype)
        self.w_x = normal(rank + 2 * states, inner)
        self.w_dt = normal(inner, rank)
        self.w_out = normal(width, inner)
        step0 = torch.exp(torch.rand(inner, device=device, generator=g) * math.log(100.0) + math.log(1e-3))
        self.dt_bias = step0 + torch.log(-torch.expm1(-step0))      # softplus(dt_bias) = step0
        self.a = -torch.arange(1, states + 1, device=device, dtype=torch.float32).repeat(inner, 1)
        self.skip = torch.ones(inner, device=device)

    def _normed(self, u):
        f = u.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-5)).to(u.dtype) * self.norm

    def _parts(self, x):
        d = la.linear(x, self.w_x)
        r, s = self.rank, self.states
        return la.linear(d[..., :r], self.w_dt), d[..., r:r + s], d[..., r + s:]

    def prefill(self, u, lengths=None, state=None):
        """u [B, n, width] → (u, state); lengths [B] int32: later tokens are padding."""
        conv_state, scan_state = state if state is not None else (None, None)
        xz = la.linear(self._normed(u), self.w_in)
        x, gate = xz[..., :self.inner], xz[..., self.inner:]
        x, conv_state = la.causal_conv(x, self.w_conv, self.b_conv, state=conv_state,
                                       lengths=lengths, return_state=True)
        dt, b, c = self._parts(x)
        y, scan_state = la.selective_scan(x, dt, self.a, b, c, skip=self.skip, gate=gate,
                                          dt_bias=self.dt_bias, state=scan_state, lengths=lengths,
                                          return_state=True)
        return la.linear(y, self.w_out, residual=u), (conv_state, scan_state)

    def step(self, u, state):
        """u [B, width], the next token → u; the state is updated in place."""
        conv_state, scan_state = state
        xz = la.linear(self._normed(u), self.w_in)
        x, gate = xz[..., :self.inner], xz[..., self.inner:]
        x = la.causal_conv_step(conv_state, x, self.w_conv, self.b_conv)
        dt, b, c = self._parts(x)
        y = la.selective_step(scan_state, x, dt, self.a, b, c, skip=self.skip, gate=gate,
                              dt_bias=self.dt_bias)
        return la.linear(y, self.w_out, residual=u)


def run(width=1024, batch=4, prompt=500, tokens=16, seed=0):
    """Prefills ragged prompts, decodes ``tokens`` inputs one by one, and returns
    the largest difference from prompts that contain them, over their size."""
    block = StateSpaceBlock(width, seed=seed)
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
    block = StateSpaceBlock(a.width)
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
