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
