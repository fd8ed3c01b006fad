"""The gated delta rule on the GPU against 64 bits, with what its kernels' parts lose.

The tolerances of test_delta_block_gpu.py add up what every token may lose.  Here they are
closer, by inputs for which little adds up, or by adding roundings that do not know of one
another as squares.
"""
import math

import pytest
import torch

import causal_kernelized_linear_gb300 as la
from test_delta_block_gpu import (BF16, CHUNKED, DEV, DTYPES, F32, IDS, LONG, SHAPES, TOKENS, U, _call, _f, _gen, _inputs,
                                  _randn, _ref)

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


# ------------------------------------------------------------------ every path, closely

def _path(x):
    """Which kernel a call takes: chunks for bf16 with dk up to 128 from 16 tokens on."""
    return CHUNKED if x["v"].dtype == BF16 and x["q"].shape[3] <= 128 and x["v"].shape[1] >= 16 else TOKENS


def _close(got, x, softplus=True, sigmoid=True, normalize=True, scale=None, state=None, lengths=None, parts=False):
    """got is (out, state) of x, held to what its kernel's roundings come to.

    One evaluation of w is off by e = f(dk) + 2^-21 of its terms in either kernel: sums of dk
    terms in fp32, whose operands keep 24 bits, and exponentials of 2 ulp.  Within 64 tokens
    these add up, E ← α·E + e·β·(‖v‖ + α‖S‖) + 2^-23‖S‖; from one chunk (or 64 tokens) to the
    next they know nothing of one another and add as squares.  So do the errors of a part's
    transition, column by column; a join adds f(dk)‖S‖.  Twice that is allowed.  An output adds
    what its operands lose: f(dk), or 2^-16 each of S, scores and values in chunks, of the
    squares' sum of what was written."""
    q, k, v, dt, beta = (x[i].double() for i in ("q", "k", "v", "dt", "beta"))
    B, n, hv, dv = v.shape
    hk, dk = q.shape[2], q.shape[3]
    scale = dk ** -0.5 if scale is None else scale
    if normalize:
        q, k = (t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
    q, k = (t.repeat_interleave(hv // hk, 2) for t in (q, k))
    d = dt if x["dt_bias"] is None else dt + x["dt_bias"].double()
    alpha = torch.exp((torch.nn.functional.softplus(d, threshold=1e9) if softplus else d) * x["a"].double())
    beta = torch.sigmoid(beta) if sigmoid else beta
    live = torch.arange(n, device=DEV) < (n if lengths is None else lengths.long()[:, None])
    live = live.expand(B, n)[..., None]
    alpha, beta = torch.where(live, alpha, 1.0), torch.where(live, beta, 0.0)
    S = torch.zeros(B, hv, dk, dv, device=DEV, dtype=torch.float64) if state is None else state.double().clone()
    norm = lambda t: t.flatten(2).norm(dim=-1)   # noqa: E731
    here, before, M = torch.zeros(B, hv, device=DEV, dtype=torch.float64), 0.0, norm(S) ** 2
    e, outs, tols = _f(dk) + 2.0 ** -21, [], []
    r = _f(dk) + (PARTS if _path(x) == CHUNKED else 0.0)
    for t in range(n):
        al, be, kt = alpha[:, t], beta[:, t], k[:, t]
        S = al[..., None, None] * S
        here = al * here + be * e * (v[:, t].norm(dim=-1) + norm(S))
        w = be[..., None] * (v[:, t] - torch.einsum("bhk,bhkv->bhv", kt, S))
        S = S + kt[..., None] * w[:, :, None]
        size = norm(S)
        here, before, M = here + live[:, t] * 2.0 ** -23 * size, al ** 2 * before, al ** 2 * M + w.norm(dim=-1) ** 2
        outs.append(torch.where(live[:, t, :, None], scale * torch.einsum("bhk,bhkv->bhv", q[:, t], S), 0.0))
        off = 2 * (before + here ** 2).sqrt() + 2 * r * torch.maximum(M.sqrt(), size)
        tols.append(torch.where(live[:, t], scale * q[:, t].norm(dim=-1) * off, 0.0))
        if t % 64 == 63:
            before, here = before + (here + parts * _f(dk) * size) ** 2, 0.0 * here
    ref, tol = torch.stack(outs, 1), torch.stack(tols, 1)
    tol = U[x["v"].dtype] * ref.norm(dim=-1) + tol + 1e-30
    off = (got[0].double() - ref).norm(dim=-1)
    assert (off <= tol).all(), f"out off by {(off / tol).max().item():.3f} of what is allowed"
    tol = 2 * (before + here ** 2).sqrt() + 1e-30
    off = norm(got[1].double() - S)
    assert (off <= tol).all(), f"state off by {(off / tol).max().item():.3f} of what is allowed"
    # what one of the parts could lose would show: entering states dropped, off by a hundredth, or in bf16
    assert (tol <= 1e-3 * norm(S) + 1e-30).all(), f"{(tol / norm(S)).max().item():.1e} of the state is allowed"


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_shapes_closely(dtype, shape):
    x = _inputs(*shape, dtype, seed=sum(shape) + 1)
    B, _, _, hv, dk, dv = shape
    state = _randn(_gen(5), B, hv, dk, dv, scale=0.3)
    _close(_call(x, state=state), x, state=state)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("n", [3, 150])
@pytest.mark.parametrize("softplus,sigmoid,normalize,bias", [
    (False, True, True, True), (True, False, True, False), (True, True, False, True), (False, False, False, False)])
def test_options_closely(dtype, n, softplus, sigmoid, normalize, bias):
    x = _inputs(2, n, 2, 4, 64, 72, dtype, seed=n + 1, gates=F32)
    if not softplus:
        x["dt"], x["dt_bias"] = x["dt"].abs() * 0.1, x["dt_bias"].abs() * 0.1
    if not sigmoid:
        x["beta"] = torch.rand(x["beta"].shape, device=DEV, generator=_gen(n))
    if not normalize:
        x["k"] = x["k"] * 0.05
    if not bias:
        x["dt_bias"] = None
    kw = {"softplus": softplus, "sigmoid": sigmoid, "normalize": normalize, "scale": 0.7}
    _close(_call(x, **kw), x, **kw)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("shape", LONG, ids=lambda s: "x".join(map(str, s[:6])))
def test_long_closely(dtype, shape):
    # walked in parts where there are few heads
    B, n, hk, hv, dk, dv, lens, with_state = shape
    x = _inputs(B, n, hk, hv, dk, dv, dtype, seed=n + 1)
    x["a"] = x["a"] * 0.002
    x["beta"] = x["beta"] - 3.0
    state = _randn(_gen(5), B, hv, dk, dv, scale=0.3) if with_state else None
    lengths = None if lens is None else torch.tensor(lens, device=DEV, dtype=torch.int32)
    got = _call(x, state=state, lengths=lengths)
    _close(got, x, state=state, lengths=lengths, parts=True)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_layouts(dtype):
    # [B, H, n, d] with its axes exchanged, gates as a part of a wider buffer
    x = _inputs(2, 100, 2, 4, 64, 64, dtype, seed=3)
    y = dict(x)
    for name in ("q", "k", "v"):
        y[name] = x[name].transpose(1, 2).contiguous().transpose(1, 2)
    for name in ("dt", "beta"):
        wide = torch.full((2, 100, 3, 11), float("nan"), device=DEV, dtype=dtype)
        wide[:, :, 1, 5:9] = x[name]
        y[name] = wide[:, :, 1, 5:9]
    for a, b in zip(_call(x), _call(y)):
        assert torch.equal(a, b)
    # gates whose heads are not next to one another are refused
    y["dt"] = x["dt"].transpose(1, 2).contiguous().transpose(1, 2)
    with pytest.raises(ValueError, match="last axis must be contiguous"):
        _call(y)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("n", [9, 100])
def test_outputs_between_values(dtype, n):
    # an output in the same buffer as the values, between them, is apart from them; on them it is refused
    B, hv, d = 2, 4, 64
    x = _inputs(B, n, 2, hv, d, d, dtype, seed=4)
    want = _call(x)
    buffers = {
        "heads": (torch.full((B, n, 3 * hv, d), 7.0, device=DEV, dtype=dtype), lambda t: t[:, :, :hv], lambda t: t[:, :, 2 * hv:]),
        "tokens": (torch.full((B, n, 2, hv, d), 7.0, device=DEV, dtype=dtype), lambda t: t[:, :, 0], lambda t: t[:, :, 1]),
        "exchanged": (torch.full((B, hv, n, 2, d), 7.0, device=DEV, dtype=dtype),
                      lambda t: t[..., 0, :].transpose(1, 2), lambda t: t[..., 1, :].transpose(1, 2)),
        "features": (torch.full((B, n, hv, 3 * d), 7.0, device=DEV, dtype=dtype), lambda t: t[..., :d], lambda t: t[..., 2 * d:])}
    for name, (buf, values, outputs) in buffers.items():
        values(buf).copy_(x["v"])
        keep = buf.clone()
        got = _call({**x, "v": values(buf)}, out=outputs(buf))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), name
        outputs(keep).copy_(want[0])
        assert torch.equal(buf, keep), name
    buf, values, _ = buffers["heads"]
    for on in (buf[:, :, :hv], buf[:, :, 2:hv + 2], buffers["features"][0][..., 8:8 + d]):
        v = values(buf) if on.stride() == values(buf).stride() else buffers["features"][0][..., :d]
        with pytest.raises(la.LinAttnError):
            _call({**x, "v": v}, out=on)
