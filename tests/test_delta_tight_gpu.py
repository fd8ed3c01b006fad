"""The gated delta rule on the GPU against 64 bits, with what its kernels' parts lose.

The tolerances of test_delta_block_gpu.py add up what every token may lose.  Here they are
closer, by inputs for which little adds up, or by adding roundings that do not know of one
another as squares.
"""
import math

import pytest
import torch

import causal_kernelized_linear_gb300 as la
from test_delta_block_gpu import BF16, DEV, DTYPES, F32, IDS, U, _f, _gen, _randn, _ref

pytestmark = pytest.mark.gpu

# What an output's parts lose in chunks: S, the scores and the corrected values are operands in
# two bf16 parts each, which keep 2^-16 of a value.
PARTS = 3 * 2.0 ** -16


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("dk", [64, 128])
def test_outputs_that_cancel(dtype, dk):
    # Two values a few tokens apart, the second the first's remains in bf16 with the sign
    # exchanged: what is read of both is what bf16 rounds away, 2^-9 of either.  Scores in one
    # bf16 part are off by as much.  No other token writes, so that M and E of the tolerance
    # stay at the two values.
    pairs = [(0, 1), (0, 15), (5, 21), (3, 36), (31, 32), (30, 63), (40, 43), (33, 60)]
    rates = [-0.011, -0.035, -0.17]
    hv = len(pairs) * len(rates)
    g = _gen(dk)
    x = {name: torch.zeros(1, 64, hv, dk, device=DEV) for name in ("q", "k")}
    x["v"] = torch.zeros(1, 64, hv, 128, device=DEV)
    x["dt"], x["beta"] = torch.ones(1, 64, hv, device=DEV), torch.zeros(1, 64, hv, device=DEV)
    x["a"], x["dt_bias"] = torch.tensor(rates * len(pairs), device=DEV), None
    for h in range(hv):
        i, j = pairs[h // len(rates)]
        for t, feature in ((i, 3), (j, 7)):
            x["k"][0, t, h, feature] = 1.0
            x["beta"][0, t, h] = 1.0
            x["q"][0, j:, h, feature] = 1.0
        v = _randn(g, 128, dtype=BF16)
        x["v"][0, i, h] = v.float()
        x["v"][0, j, h] = -(math.exp((j - i) * x["a"][h].item()) * v.double()).to(BF16).float()
    for name in ("q", "k", "v"):
        x[name] = x[name].to(dtype)
    kw = {"softplus": False, "sigmoid": False, "normalize": False, "scale": 1.0}
    out, state = la.gated_delta(x["q"], x["k"], x["v"], x["dt"], x["a"], x["beta"], return_state=True, **kw)
    ref, _, tols, _ = _ref(x, **kw)
    chunked = dtype == BF16
    e = _f(dk) + (4 * 2.0 ** -16 if chunked else 0.0)
    r = _f(dk) + (PARTS if chunked else 0.0)
    off = (out.double() - ref).norm(dim=-1)
    tol = U[dtype] * ref.norm(dim=-1) + e * tols[0] + tols[1] + r * tols[2] + 1e-30
    assert (off <= tol).all(), f"off by {(off / tol).max().item():.2f} of what is allowed"


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("n", [20, 64, 100])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("writes", [1, 2])
def test_single_writes_keep_24_bits(dtype, n, dk, writes):
    # Keys with one feature each, a different one at every token that writes (or at every two):
    # a row of S is then (1 − β)αS + βv, with nothing to sum, and is held to 2^-19 of its terms
    # (two exponentials of 2 ulp each, some twenty roundings and cut-off sums of 2^-24).
    # Operands of 16 bits, two bf16 parts, would be off by up to 2^-17 each.  Token by token (fp32)
    # every token rounds S once more, by 2^-24 of it: α and the product, whatever is written.
    B, hv, dv = 2, 3, 128
    g = _gen(n + dk)
    at = torch.randperm(n, device=DEV, generator=g)[:min(n // 2, dk) // writes * writes]
    row = torch.randperm(dk, device=DEV, generator=g)[:at.numel() // writes].repeat(writes)
    x = {"q": torch.zeros(B, n, hv, dk, device=DEV, dtype=dtype), "k": torch.zeros(B, n, hv, dk, device=DEV, dtype=dtype),
         "v": _randn(g, B, n, hv, dv, dtype=dtype), "dt": torch.rand(B, n, hv, device=DEV, generator=g) * 0.1,
         "beta": torch.zeros(B, n, hv, device=DEV), "a": torch.tensor([0.0, -0.3, -2.0], device=DEV), "dt_bias": None}
    x["v"][0] = 0   # what is left of a state alone, and of values written over it
    x["k"][:, at, :, row] = 1.0
    x["beta"][:, at] = torch.rand(B, at.numel(), hv, device=DEV, generator=g)
    state = _randn(g, B, hv, dk, dv)
    kw = {"softplus": False, "sigmoid": False, "normalize": False, "scale": 1.0, "state": state}
    _, got = la.gated_delta(x["q"], x["k"], x["v"], x["dt"], x["a"], x["beta"], return_state=True, **kw)
    S = state.double()
    terms = S.abs()   # what a row was made of, decayed
    alpha = torch.exp(x["dt"].double() * x["a"].double())
    for t in range(n):
        al, be = alpha[:, t][..., None, None], x["beta"][:, t].double()[..., None, None] * x["k"][:, t].double()[..., None]
        v = x["v"][:, t].double()[:, :, None]
        S = al * S
        S = S + be * (v - S)
        terms = al * terms + be * v.abs()
    tol = (2.0 ** -19 + (n * 2.0 ** -24 if dtype == F32 else 0.0)) * terms + 1e-30
    off = (got.double() - S).abs()
    assert (off <= tol).all(), f"off by {(off / tol).max().item():.2f} of what is allowed"


def _slow(n, x):
    """How far n roundings of 2^-24 take a state that decays by e^x (x < 0) at each, relative to
    it and in the root mean square of its elements, twice over.  They are as good as independent
    but for runs in which what is taken off lies alike between two values of fp32: it is
    |x|·2^23 to 2^24 steps, and shrinks by |x| of that from one time to the next.  An exponent's
    roundings are 2^-23 of it, four of them."""
    run = max(1.0, 1 / (x * x * 2.0 ** 23))
    return 2 * 2.0 ** -24 * math.sqrt(n * run) + 4 * 2.0 ** -23 * -x * n


SLOW = [(3000, 1e-3, -1.0), (30000, 1e-3, -0.1), (65536, 1e-3, -0.016)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("hv,n,dt,a", [(1, *s) for s in SLOW] + [(1300, *SLOW[0])])   # in parts; undivided
def test_slow_decays(dtype, hv, n, dt, a):
    # nothing is written: the state is decayed n times by factors next to 1
    d = 32
    state = _randn(_gen(n), 1, hv, d, d)
    zero = torch.zeros(1, n, 1, d, device=DEV, dtype=dtype)
    step = torch.full((1, n, hv), dt, device=DEV)
    _, got = la.gated_delta(zero, zero, zero.expand(1, n, hv, d), step, torch.full((hv,), a, device=DEV),
                            torch.zeros_like(step), softplus=False, sigmoid=False, state=state, return_state=True)
    x = step[0, 0, 0].double() * float(torch.tensor(a))
    want = state.double() * torch.exp(n * x)
    off = ((got.double() - want).norm() / want.norm()).item()
    chunks = (n + 63) // 64
    tol = _slow(chunks, 64 * x.item()) if dtype == BF16 else _slow(n, x.item())
    assert off <= tol, f"off by {off:.2e} where {tol:.2e} is allowed"


@pytest.mark.parametrize("dk", [64, 128, 256])
def test_slow_decays_step_by_step(dk):
    n, dt, a = SLOW[0]
    state = _randn(_gen(n), 1, 2, dk, 64)
    start = state.clone()
    zero = torch.zeros(1, 2, dk, device=DEV)
    step, rate = torch.full((1, 2), dt, device=DEV), torch.full((2,), a, device=DEV)
    v, none = zero[..., :64].contiguous(), torch.zeros_like(step)
    for _ in range(n):
        la.gated_delta_step(state, zero, zero, v, step, rate, none, softplus=False, sigmoid=False)
    x = step[0, 0].double() * a
    want = start.double() * torch.exp(n * x)
    off = ((state.double() - want).norm() / want.norm()).item()
    assert off <= _slow(n, x.item()), f"off by {off:.2e}"
