"""Gated-delta block operators on the GPU against plain 64-bit forms.

Tolerances.  u = eps/2 of a type (bf16 2^-8, fp32 2^-24, e4m3 2^-4).  Sums of N
terms in fp32 are allowed f(N) = (2·sqrt(N) + 16)·2^-24 of the sum of their
absolute values, as for the state-space block's operators.

The gated delta rule S ← α(1 − β kᵀk)S + kᵀβv with ‖k‖ ≤ 1 and β ≤ 1 does not
enlarge an error of S, so what is added per token is bounded by
  E ← α·E + e·β·(‖v‖ + α‖S‖) + 2^-23·‖S‖          (Frobenius norms)
where e is what one evaluation of v − k·S may be off by, relative to its terms:
  * token by token in fp32: f(dk);
  * in chunks on the tensor cores: S, the chunk's inverse and the corrected values
    go in as two bf16 parts, which keep 2^-16 of a value; four such operands
    meet (S; the inverse and k·S; the values), 4·2^-16 + f(dk).
With M ← α·M + ‖w‖ (M starts at ‖S_0‖), which bounds the norm of every partial
sum that q·S is made of, an output row is off by at most
  u·‖o‖ + scale·‖q‖·(E + r·M),  r = f(dk), or 3·2^-8 where S, the chunk's
scores and its values are rounded to bf16 for the output alone.

A long sequence of few heads is walked in parts, S ← Φ·S + N over one, where Φ
is what a part makes of the identity and N of a zero state.  A column of Φ has a
norm of at most the part's decay D, D‖S‖ ≤ M, and ‖N‖ ≤ ‖S'‖ + D‖S‖ ≤ 2M.  What a
token adds to Φ's error, e·β·α·D per column, meets ‖S‖ by way of Φ's Frobenius norm,
√dk times as much, so √dk·αM stands in for α‖S‖ above (dk ≥ 8 covers N's 2M).  The
product and the sum of a join in fp32 are off by f(dk)·‖Φ‖‖S‖ ≤ f(dk)·√dk·M each, which
decays as M does: there are at most 63 joins, 32 tokens or more apart.
"""
import importlib.util
import math
import os
import subprocess
import sys

import pytest
import torch

import causal_kernelized_linear_gb300 as la

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24, E4M3: 2.0 ** -4}
DTYPES = [BF16, F32]
IDS = ["bf16", "f32"]


def _f(n):
    return (2 * math.sqrt(n) + 16) * 2.0 ** -24


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, device=DEV, generator=g) * scale).to(dtype)


# ------------------------------------------------------------------ gated delta rule

def _inputs(B, n, hk, hv, dk, dv, dtype, seed, skew=True, gates=None):
    g = _gen(seed)
    qkv = _randn(g, B, n, 2 * hk * dk + hv * dv, dtype=F32)
    if skew:   # as behind a silu: keys that resemble each other
        qkv = qkv * torch.sigmoid(qkv)
    q, k, v = qkv.to(dtype).split([hk * dk, hk * dk, hv * dv], -1)
    db = _randn(g, B, n, 2 * hv, dtype=gates or dtype)
    return {"q": q.unflatten(-1, (hk, dk)), "k": k.unflatten(-1, (hk, dk)), "v": v.unflatten(-1, (hv, dv)),
            "dt": db[..., :hv], "beta": db[..., hv:],
            "a": -torch.rand(hv, device=DEV, generator=g) * 4.0,
            "dt_bias": _randn(g, hv) - 1.0}


def _ref(x, softplus=True, sigmoid=True, normalize=True, scale=None, state=None, lengths=None, parts=False):
    """(out, state, error of an output row apart from its own rounding, error of the
    state per head) from the recurrence in 64 bits; the errors for e = r = 1."""
    q, k, v, dt, beta = (x[i].double() for i in ("q", "k", "v", "dt", "beta"))
    B, n, hv, dv = v.shape
    hk, dk = q.shape[2], q.shape[3]
    scale = dk ** -0.5 if scale is None else scale
    if normalize:
        q = q / (q.square().sum(-1, keepdim=True) + 1e-6).sqrt()
        k = k / (k.square().sum(-1, keepdim=True) + 1e-6).sqrt()
    q, k = (t.repeat_interleave(hv // hk, 2) for t in (q, k))
    d = dt if x["dt_bias"] is None else dt + x["dt_bias"].double()
    d = torch.nn.functional.softplus(d, threshold=1e9) if softplus else d
    alpha = torch.where(d == 0, 1.0, torch.exp(d * x["a"].double()))
    beta = torch.sigmoid(beta) if sigmoid else beta
    S = torch.zeros(B, hv, dk, dv, device=v.device, dtype=torch.float64) if state is None else state.double().clone()
    norm = lambda t: t.flatten(2).norm(dim=-1)   # noqa: E731
    E = [torch.zeros(B, hv, device=v.device, dtype=torch.float64) for _ in range(2)]   # for e, and for rounding S
    M = norm(S)
    out = torch.zeros(B, n, hv, dv, device=v.device, dtype=torch.float64)
    tols = torch.zeros(3, B, n, hv, device=v.device, dtype=torch.float64)
    lens = torch.full((B,), n, device=v.device) if lengths is None else lengths.long().clamp(0, n)
    for t in range(n):
        live = (t < lens)[:, None]
        al = torch.where(live, alpha[:, t], 1.0)
        be = torch.where(live, beta[:, t], 0.0)
        kt = torch.where(live[..., None], k[:, t], 0.0)   # what is not read may be anything
        vt = torch.where(live[..., None], v[:, t], 0.0)
        S = al[..., None, None] * S
        before = al * M * dk ** 0.5 if parts else norm(S)
        w = be[..., None] * (vt - torch.einsum("bhk,bhkv->bhv", kt, S))
        S = S + kt[..., None] * w[:, :, None]
        E[0] = al * E[0] + be * (vt.norm(dim=-1) + before)
        E[1] = al * E[1] + live * 2.0 ** -23 * norm(S)
        M = al * M + w.norm(dim=-1)
        o = scale * torch.einsum("bhk,bhkv->bhv", q[:, t], S)
        out[:, t] = torch.where(live[..., None], o, 0.0)
        s = scale * q[:, t].norm(dim=-1)
        joins = min(63, t // 32) * dk ** 0.5 * _f(dk) * M if parts else 0.0
        tols[:, :, t] = torch.where(live, s * torch.stack([E[0], E[1] + joins, M]), 0.0)
    if parts:
        E[1] = E[1] + joins
    return out, S, tols, torch.stack(E)


CHUNKED, TOKENS = "chunked", "tokens"


def _check(got, x, how=CHUNKED, what="", **kw):
    """got is (out, state) of x; `how` is what the tolerance allows for."""
    ref, S, tols, E = _ref(x, **kw)
    out, state = got
    dk, dtype = x["q"].shape[3], x["v"].dtype
    chunked = how == CHUNKED
    e = (4 * 2.0 ** -16 if chunked else 0.0) + _f(dk)
    r = 3 * 2.0 ** -8 if chunked and dtype == BF16 else e
    assert out.dtype == dtype and out.shape == ref.shape and state.dtype == F32
    assert torch.isfinite(out).all() and torch.isfinite(state).all(), what
    off = (out.double() - ref).norm(dim=-1)
    tol = U[dtype] * ref.norm(dim=-1) + e * tols[0] + tols[1] + r * tols[2] + 1e-30
    assert (off <= tol).all(), f"{what}: out off by {(off / tol).max().item():.3f} of what is allowed"
    off = (state.double() - S).flatten(2).norm(dim=-1)
    tol = e * E[0] + E[1] + 1e-30
    assert (off <= tol).all(), f"{what}: state off by {(off / tol).max().item():.3f} of what is allowed"


def _call(x, **kw):
    return la.gated_delta(x["q"], x["k"], x["v"], x["dt"], x["a"], x["beta"], dt_bias=x["dt_bias"],
                          return_state=True, **kw)


SHAPES = [  # B, n, hk, hv, dk, dv
    (1, 1, 1, 1, 8, 8), (2, 2, 1, 2, 64, 64), (1, 37, 2, 4, 128, 128), (3, 63, 1, 1, 96, 192), (1, 64, 2, 2, 128, 128),
    (2, 65, 1, 4, 64, 128), (1, 127, 3, 3, 72, 40), (1, 128, 1, 2, 128, 256), (2, 129, 2, 2, 128, 136),
    (1, 191, 1, 1, 40, 8), (1, 200, 1, 1, 256, 512), (2, 333, 2, 4, 128, 128), (1, 515, 1, 1, 16, 128),
    (1, 1000, 2, 2, 128, 64), (5, 77, 3, 9, 136, 72)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("with_state", [False, True])
def test_gated_delta_shapes(dtype, shape, with_state):
    x = _inputs(*shape, dtype, seed=sum(shape))
    B, _, _, hv, dk, dv = shape
    state = _randn(_gen(5), B, hv, dk, dv, scale=0.3) if with_state else None
    got = _call(x, state=state)
    _check(got, x, state=state)
    again = _call(x, state=state)   # a fixed order of sums
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("n", [3, 150])
@pytest.mark.parametrize("softplus,sigmoid,normalize,bias", [
    (False, True, True, True), (True, False, True, False), (True, True, False, True), (False, False, False, False)])
def test_gated_delta_options(dtype, n, softplus, sigmoid, normalize, bias):
    x = _inputs(2, n, 2, 4, 64, 72, dtype, seed=n, gates=F32)
    if not softplus:   # steps as they are
        x["dt"] = x["dt"].abs() * 0.1
        x["dt_bias"] = x["dt_bias"].abs() * 0.1
    if not sigmoid:
        x["beta"] = torch.rand(x["beta"].shape, device=DEV, generator=_gen(n))
    if not normalize:   # keys within the unit ball
        x["k"] = x["k"] * 0.05
    if not bias:
        x["dt_bias"] = None
    kw = {"softplus": softplus, "sigmoid": sigmoid, "normalize": normalize, "scale": 0.7}
    _check(_call(x, **kw), x, **kw)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("lens", [[0, 1, 64, 200, 199, 65], [-3, 500, 63, 128, 127, 0]])
def test_gated_delta_lengths(dtype, lens):
    B, n = len(lens), 200
    x = _inputs(B, n, 1, 2, 128, 64, dtype, seed=9)
    state = _randn(_gen(6), B, 2, 128, 64, scale=0.3)
    lengths = torch.tensor(lens, device=DEV, dtype=torch.int32)
    for i, l in enumerate(lens):   # what lies behind a sequence is not read
        for name in ("q", "k", "v", "dt", "beta"):
            x[name][i, max(0, min(n, l)):] = float("nan")
    got = _call(x, state=state, lengths=lengths)
    clean = dict(x)
    for name in ("q", "k", "v", "dt", "beta"):
        clean[name] = torch.nan_to_num(x[name])
    _check(got, clean, state=state, lengths=lengths)
    assert torch.equal(got[1][0], state[0])
    for i, l in enumerate(lens):
        assert (got[0][i, max(0, l):] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gated_delta_views(dtype):
    # [B, H, n, d] tensors with their axes exchanged, outputs in the middle of a buffer
    x = _inputs(2, 100, 2, 4, 64, 64, dtype, seed=3)
    y = dict(x)
    for name in ("q", "k", "v"):
        y[name] = x[name].transpose(1, 2).contiguous().transpose(1, 2)
    y["dt"] = x["dt"].transpose(1, 2).contiguous().transpose(1, 2)[:, :, :]
    y["dt"] = torch.stack([x["dt"]] * 3, 1)[:, 1]
    ref = _call(x)
    got = _call(y)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    big = _randn(_gen(4), 2, 102, 6, 80, dtype=dtype)
    keep = big.clone()
    out = big[:, 1:101, 1:5, 8:72]
    got = _call(x, out=out)
    assert got[0].data_ptr() == out.data_ptr() and torch.equal(out, ref[0])
    big[:, 1:101, 1:5, 8:72] = keep[:, 1:101, 1:5, 8:72]
    assert torch.equal(big, keep)
    # the same keys and values for every sequence of a batch
    for name in ("q", "k", "v", "dt", "beta"):
        y[name] = x[name][:1].expand(2, *x[name].shape[1:])
    got = _call(y)
    assert torch.equal(got[0][0], got[0][1]) and torch.equal(got[0][0], ref[0][0])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gated_delta_broadcast_axes(dtype):
    # one key and query for all heads, one token for all, and rows that overlap
    x = _inputs(2, 100, 2, 4, 64, 64, dtype, seed=3)
    y = dict(x)
    for name in ("q", "k"):
        y[name] = x[name][:, :, :1].expand(2, 100, 2, 64)
    z = {k: (v.contiguous() if v.dim() > 1 else v) for k, v in y.items()}
    for a, b in zip(_call(y), _call(z)):
        assert torch.equal(a, b)
    y["v"] = x["v"][:, :1].expand(2, 100, 4, 64)
    y["dt"], y["beta"] = (x[i][:, :1].expand(2, 100, 4) for i in ("dt", "beta"))
    _check(_call(y), y)
    line = x["v"].flatten()
    y["v"] = line.as_strided((2, 100, 4, 64), (4096, 16, 8, 1))
    z["v"] = y["v"].contiguous()
    y["dt"], y["beta"] = z["dt"], z["beta"]
    for a, b in zip(_call(y), _call(z)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gated_delta_extreme_decays(dtype):
    # no decay at all, decays that clear the state, and steps of zero
    x = _inputs(1, 260, 2, 4, 64, 64, dtype, seed=8, gates=F32)
    x["a"] = torch.tensor([0.0, -1e4, float("-inf"), -30.0], device=DEV)
    x["dt_bias"] = None
    x["dt"] = torch.rand(x["dt"].shape, device=DEV, generator=_gen(1))
    x["dt"][:, ::3] = 0.0
    state = _randn(_gen(2), 1, 4, 64, 64)
    _check(_call(x, softplus=False, state=state), x, softplus=False, state=state)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gated_delta_equal_keys(dtype):
    # the same unit key at every token, full strength: each token replaces what the one before wrote
    x = _inputs(1, 200, 1, 1, 64, 64, dtype, seed=8, gates=F32)
    x["k"] = torch.zeros_like(x["k"])
    x["k"][..., 5] = 1.0
    x["q"] = x["k"].clone()
    x["a"].zero_()
    x["beta"] = torch.ones_like(x["beta"])
    kw = {"sigmoid": False, "normalize": False, "scale": 1.0}
    got = _call(x, **kw)
    _check(got, x, **kw)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gated_delta_keeps_nan_in_its_head(dtype):
    x = _inputs(2, 150, 2, 2, 64, 64, dtype, seed=2)
    ref = _call(x)
    x["v"][0, 70, 1, 3] = float("nan")
    out, state = _call(x)
    assert torch.equal(out[1], ref[0][1]) and torch.equal(out[0, :, 0], ref[0][0, :, 0])
    assert torch.equal(out[0, :64, 1], ref[0][0, :64, 1])
    assert torch.isnan(out[0, 70:, 1, 3]).all() and torch.isnan(state[0, 1, :, 3]).all()
    assert torch.equal(state[0, 0], ref[1][0, 0]) and torch.equal(state[1], ref[1][1])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gated_delta_empty(dtype):
    x = _inputs(2, 4, 1, 2, 64, 64, dtype, seed=2)
    none = {k: (v[:, :0] if v.dim() > 1 else v) for k, v in x.items()}
    state = _randn(_gen(2), 2, 2, 64, 64)
    out, after = _call(none, state=state)
    assert out.shape == (2, 0, 2, 64) and torch.equal(after, state)
    assert (_call(none)[1] == 0).all()
    out, after = _call({k: (v[:0] if v.dim() > 1 else v) for k, v in x.items()})
    assert out.shape == (0, 4, 2, 64) and after.shape == (0, 2, 64, 64)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gated_delta_in_parts(dtype):
    # a prompt in three calls, and its last tokens one by one
    n, cuts = 300, (0, 64, 171, 296)
    x = _inputs(2, n, 1, 2, 128, 128, dtype, seed=4)
    part = lambda lo, hi: {k: (v[:, lo:hi] if v.dim() > 1 else v) for k, v in x.items()}   # noqa: E731
    state, outs = None, []
    for lo, hi in zip(cuts, cuts[1:]):
        out, state = _call(part(lo, hi), state=state)
        outs.append(out)
    for t in range(cuts[-1], n):
        outs.append(la.gated_delta_step(state, x["q"][:, t], x["k"][:, t], x["v"][:, t], x["dt"][:, t], x["a"],
                                        x["beta"][:, t], dt_bias=x["dt_bias"])[:, None])
    _check((torch.cat(outs, 1), state), x)


LONG = [  # B, n, hk, hv, dk, dv, lengths, state; few heads, which are walked in parts where dk allows
    (1, 4000, 1, 1, 128, 128, None, False), (2, 2051, 1, 2, 64, 192, [2051, 700], True),
    (1, 2900, 2, 2, 72, 40, None, True), (3, 2500, 1, 1, 128, 136, [0, 1, 2499], True),
    (2, 2304, 1, 1, 128, 64, [1088, 1153], False), (1, 900, 1, 1, 256, 64, None, True),
    (7, 340, 4, 8, 64, 128, [340, 0, 1, 100, 339, 57, 200], True)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("shape", LONG, ids=lambda s: "x".join(map(str, s[:6])))
def test_gated_delta_long(dtype, shape):
    B, n, hk, hv, dk, dv, lens, with_state = shape
    x = _inputs(B, n, hk, hv, dk, dv, dtype, seed=n)
    x["a"] = x["a"] * 0.002   # the state lasts for thousands of tokens
    x["beta"] = x["beta"] - 3.0
    state = _randn(_gen(5), B, hv, dk, dv, scale=0.3) if with_state else None
    lengths = None if lens is None else torch.tensor(lens, device=DEV, dtype=torch.int32)
    kw = {"state": state, "lengths": lengths}
    big = torch.full((B, n + 2, hv, dv), 7.0, device=DEV, dtype=dtype)
    got = _call(x, out=big[:, 1:-1], **kw)
    _check(got, x, parts=True, **kw)
    assert (big[:, 0] == 7).all() and (big[:, -1] == 7).all()
    again = _call(x, **kw)   # a fixed order of sums
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    # the same beside many more heads, where nothing is divided: both within their tolerance
    wide = {k: (v.repeat(160 // B, *[1] * (v.dim() - 1)) if v.dim() > 1 else v) for k, v in x.items()}
    whole = _call(wide, state=None if state is None else state.repeat(160 // B, 1, 1, 1),
                  lengths=None if lens is None else lengths.repeat(160 // B))
    assert torch.equal(whole[1][:B], whole[1][-B:])
    _check((whole[0][:B], whole[1][:B]), x, **kw)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gated_delta_long_graph(dtype):
    # parts in captured graphs, which have their workspaces of their own, and NaN in one head of one part
    x = _inputs(1, 2500, 1, 2, 64, 64, dtype, seed=3)
    x["a"] = x["a"] * 0.002
    fixed = {k: v.clone() for k, v in x.items()}
    ref = _call(x)
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            outs.append(_call(fixed))
        graphs.append(graph)
    fixed["v"][0, 1500, 1, 3] = float("nan")
    for graph in graphs:
        graph.replay()
    for out, state in outs:
        assert torch.equal(out[:, :, 0], ref[0][:, :, 0]) and torch.equal(state[:, 0], ref[1][:, 0])
        assert torch.equal(out[0, :1437, 1], ref[0][0, :1437, 1])
        assert torch.isnan(out[0, 1500:, 1, 3]).all() and torch.isnan(state[0, 1, :, 3]).all()
        rest = [i for i in range(64) if i != 3]
        assert torch.isfinite(state[0, 1][:, rest]).all()
    fixed["v"].copy_(x["v"])
    for graph in graphs:
        graph.replay()
    for out, state in outs:
        assert torch.equal(out, ref[0]) and torch.equal(state, ref[1])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("n", [14, 15, 16, 17, 18, 31, 33])
def test_gated_delta_few_tokens(dtype, n):
    x = _inputs(2, n, 1, 2, 128, 128, dtype, seed=n)
    state = _randn(_gen(5), 2, 2, 128, 128, scale=0.3)
    _check(_call(x, state=state), x, state=state)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 72), (40, 64)])
def test_gated_delta_few_tokens_of_many_heads(dtype, dk, dv):
    x = _inputs(20, 9, 4, 16, dk, dv, dtype, seed=dk)
    lengths = torch.arange(-5, 15, device=DEV, dtype=torch.int32)
    state = _randn(_gen(5), 20, 16, dk, dv, scale=0.3)
    _check(_call(x, state=state, lengths=lengths), x, how=TOKENS, state=state, lengths=lengths)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("B,hk,hv,dk,dv", [(1, 1, 1, 8, 8), (1, 2, 4, 128, 128), (3, 1, 3, 64, 192), (2, 2, 2, 256, 40),
                                           (65, 2, 8, 128, 128), (2, 1, 1, 120, 512)])
def test_gated_delta_step(dtype, B, hk, hv, dk, dv):
    x = _inputs(B, 3, hk, hv, dk, dv, dtype, seed=B + dk)
    state = _randn(_gen(6), B, hv, dk, dv, scale=0.3)
    start, outs = state.clone(), []
    for t in range(3):
        out = torch.empty(B, hv, dv, device=DEV, dtype=dtype) if t == 1 else None
        outs.append(la.gated_delta_step(state, x["q"][:, t], x["k"][:, t], x["v"][:, t], x["dt"][:, t], x["a"],
                                        x["beta"][:, t], dt_bias=x["dt_bias"], out=out))
        assert out is None or outs[-1].data_ptr() == out.data_ptr()
    _check((torch.stack(outs, 1), state), x, how=TOKENS, state=start)


# ------------------------------------------------------------------ norm

def _norm_ref(x, weight, group, eps, gate, residual):
    """(y, the sum of the absolute parts of its error in units of 2^-24·f, h)."""
    h = x.double() if residual is None else x.double() + residual.double()
    g = h.unflatten(-1, (-1, group))
    y = g / (g.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * weight.double()
    y = y.flatten(-2)
    if gate is not None:
        y = y * gate.double() * torch.sigmoid(gate.double())
    return y, h


def _norm_close(got, x, weight, group, eps, gate, residual, quantize):
    y, h = _norm_ref(x, weight, group, eps, gate, residual)
    got = got if isinstance(got, tuple) else (got,)
    assert len(got) == 1 + quantize + (residual is not None)
    # relative error before the last rounding: half the sum's, rsqrt's two steps, three
    # products, the residual's addition, and silu's (1.25·|g| + 9) steps
    rel = _f(group) / 2 + 8 * 2.0 ** -24
    tol = rel * y.abs()
    if residual is not None:   # an addition that cancels is off by a step of its operands
        w = 1.0 if weight is None else weight.double().abs().max()
        s = 1.0 if gate is None else gate.double().abs().max()
        tol = tol + 2.0 ** -24 * h.abs() * w * s / eps ** 0.5
    if gate is not None:
        tol = tol + (1.25 * gate.double().abs() + 9) * 2.0 ** -24 * y.abs() + 1.2e-36
    if quantize:
        out, scale = got[0], got[1]
        assert out.dtype == E4M3 and scale.shape == x.shape[:-1] and scale.dtype == F32
        most = y.abs().amax(-1)
        want = torch.where(most == 0, 1.0, most / 448)
        assert ((scale.double() - want).abs() <= (tol.amax(-1) / 448 + 2.0 ** -23 * want)).all()
        val = out.double() * scale.double()[..., None]
        # half a step of 8 bits, whose steps stop shrinking at 2^-6: 2^-10 of the scale there
        tol = tol + U[E4M3] * y.abs() * (1 + 2.0 ** -20) + 2.0 ** -10 * scale.double()[..., None] + tol.amax(-1, keepdim=True)
        assert ((val - y).abs() <= tol).all(), ((val - y).abs() - tol).max()
    else:
        assert got[0].dtype == x.dtype
        tol = tol + U[x.dtype] * y.abs() + 1e-30
        assert ((got[0].double() - y).abs() <= tol).all(), ((got[0].double() - y).abs() - tol).max()
    if residual is not None:
        assert torch.equal(got[-1], (x.float() + residual.float()).to(x.dtype))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("m,d,group", [
    (1, 8, 8), (3, 64, 64), (5, 1000, 1000), (7, 2048, 2048), (2, 2056, 2056), (130, 4096, 128), (9, 512, 64), (4, 360, 72),
    (3, 4096, 512), (2, 8192, 8192), (2, 16384, 16384), (1, 32768, 32768), (33, 256, 8), (2, 24576, 1536)])
@pytest.mark.parametrize("gated,added,quantize", [(False, False, False), (True, False, False), (False, True, True),
                                                  (True, True, True), (False, True, False)])
def test_rms_norm_shapes(dtype, m, d, group, gated, added, quantize):
    g = _gen(m + d)
    x = _randn(g, m, d, dtype=dtype, scale=2.0)
    weight = _randn(g, group, dtype=dtype)
    gate = _randn(g, m, 2 * d, dtype=dtype)[:, d:] if gated else None
    residual = _randn(g, m, d, dtype=dtype) if added else None
    got = la.rms_norm(x, weight, gate=gate, residual=residual, quantize=quantize)
    _norm_close(got, x, weight, group, 1e-6, gate, residual, quantize)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_rms_norm_rows(dtype):
    # rows of zeros, of one value, of tiny and huge ones; and no weight
    d = 264
    x = torch.zeros(6, d, device=DEV, dtype=dtype)
    x[1] = 3.0
    x[2, 7] = 1e4
    x[3] = 1e-18
    x[4] = 1e17 * _randn(_gen(1), d).to(dtype)
    for quantize in (False, True):
        got = la.rms_norm(x, quantize=quantize, eps=1e-5)
        _norm_close(got, x, None, d, 1e-5, None, None, quantize)
    out, scale = la.rms_norm(x, quantize=True)
    assert (out[0].float() == 0).all() and scale[0].item() == 1.0
    assert out.float().abs().amax(-1).tolist()[1:5] == [448.0] * 4
    y = la.rms_norm(x, group=88)
    _norm_close(y, x, None, 88, 1e-6, None, None, False)


@pytest.mark.parametrize("quantize", [False, True])
def test_rms_norm_keeps_nan_in_its_row(quantize):
    x = _randn(_gen(3), 5, 512, dtype=BF16)
    ref = la.rms_norm(x, quantize=True) if quantize else (la.rms_norm(x),)
    x[2, 100] = float("nan")
    got = la.rms_norm(x, quantize=True) if quantize else (la.rms_norm(x),)
    for a, b in zip(got, ref):
        a, b = a.float(), b.float()
        assert torch.isnan(a[2]).all()
        assert torch.equal(a[[0, 1, 3, 4]], b[[0, 1, 3, 4]])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_rms_norm_in_place_and_views(dtype):
    g = _gen(11)
    big = _randn(g, 4, 9, 200, dtype=dtype)
    x, residual = big[..., 16:152], _randn(g, 4, 9, 136, dtype=dtype)
    weight = _randn(g, 136, dtype=dtype)
    want, total = la.rms_norm(x, weight, residual=residual)
    keep = big.clone()
    a, b = residual.clone(), x
    out, s = la.rms_norm(b, weight, residual=a, out=b, sum_out=a)
    assert out.data_ptr() == x.data_ptr() and s.data_ptr() == a.data_ptr()
    assert torch.equal(out, want) and torch.equal(s, total)
    keep[..., 16:152] = want
    assert torch.equal(big, keep)
    gate = _randn(g, 36, 136, dtype=dtype)
    want = la.rms_norm(residual.view(36, 136), weight, gate=gate)
    assert torch.equal(la.rms_norm(residual.view(36, 136), weight, gate=gate, out=gate), want)
    assert la.rms_norm(x[:, :0], weight).shape == (4, 0, 136)
    out, scale = la.rms_norm(x[:0], weight, quantize=True)
    assert out.shape == (0, 9, 136) and scale.shape == (0, 9)


# ------------------------------------------------------------------ product of 8-bit operands

ACTS = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v * torch.sigmoid(v),
        "gelu": lambda v: v * torch.special.ndtr(v), "softplus": lambda v: torch.logaddexp(v, torch.zeros_like(v))}


def _linear8(m, k, n, seed, bias=True, residual=True):
    g = _gen(seed)
    x, w = (_randn(g, m, k, scale=40.0).to(E4M3), _randn(g, n, k, scale=60.0).to(E4M3))
    xs, ws = torch.rand(m, device=DEV, generator=g) * 0.05, torch.rand(n, device=DEV, generator=g) * 0.02 * k ** -0.5
    return (x, xs, w, ws, _randn(g, n, dtype=BF16) if bias else None,
            _randn(g, m, n, dtype=BF16) if residual else None)


def _linear8_close(y, x, xs, w, ws, bias, residual, act="none"):
    f = lambda t: t.double()   # noqa: E731
    s = f(xs)[:, None] * f(ws)
    ref, ab = f(x) @ f(w).t() * s, f(x).abs() @ f(w).abs().t() * s
    if bias is not None:
        ref, ab = ref + f(bias), ab + f(bias).abs()
    ref, ab = ACTS[act](ref), 1.13 * ab + 1.0
    if residual is not None:
        ref, ab = ref + f(residual), ab + f(residual).abs()
    # the fp32 sum's order is the tensor core's: its terms are aligned to the largest of a
    # group and cut there, up to two steps of 2^-24 each
    tol = U[BF16] * ref.abs() + 2 * _f(x.shape[1] + 4) * ab + 1e-30
    assert y.dtype == BF16 and ((y.double() - ref).abs() <= tol).all(), ((y.double() - ref).abs() - tol).max()


@pytest.mark.parametrize("m,k,n", [
    (1, 16, 8), (1, 4096, 264), (2, 128, 8), (7, 144, 136), (16, 2048, 520), (33, 400, 1000), (64, 256, 128), (65, 128, 72),
    (127, 96, 256), (128, 512, 384), (129, 1040, 264), (255, 64, 2048), (256, 256, 256), (257, 1040, 520), (700, 48, 8),
    (1000, 16, 1032), (2049, 144, 264), (5000, 80, 640)])
def test_linear_e4m3_shapes(m, k, n):
    args = _linear8(m, k, n, m * 7 + k * 3 + n)
    x, xs, w, ws, bias, residual = args
    y = la.linear_e4m3(x, xs, w, ws, bias=bias, residual=residual)
    _linear8_close(y, *args)
    assert torch.equal(y, la.linear_e4m3(x, xs, w, ws, bias=bias, residual=residual))


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("m", [3, 40, 300])
@pytest.mark.parametrize("use_bias,use_res", [(False, False), (True, False), (False, True)])
def test_linear_e4m3_epilogues(act, m, use_bias, use_res):
    args = _linear8(m, 160, 328, m, use_bias, use_res)
    x, xs, w, ws, bias, residual = args
    _linear8_close(la.linear_e4m3(x, xs, w, ws, bias=bias, activation=act, residual=residual), *args, act=act)


@pytest.mark.parametrize("m", [1, 5, 200, 1025])
def test_linear_e4m3_views(m):
    x, xs, w, ws, _, _ = _linear8(m, 112, 139, m, False, False)
    x, w, ws = x[:, 16:96], w[2:138, 32:], ws[:136].clone()
    big = _randn(_gen(m), m, 184, dtype=BF16)
    keep, out = big.clone(), big[:, 16:152]
    res = out.clone()
    got = la.linear_e4m3(x, xs, w, ws, activation="relu", residual=out, out=out)
    assert got.data_ptr() == out.data_ptr()
    _linear8_close(got, x, xs, w, ws, None, res, act="relu")
    assert torch.equal(big[:, :16], keep[:, :16]) and torch.equal(big[:, 152:], keep[:, 152:])
    lead = la.linear_e4m3(x.unflatten(0, (1, m)), xs[None], w, ws)
    assert lead.shape == (1, m, 136)
    assert la.linear_e4m3(x[:0], xs[:0], w, ws).shape == (0, 136)


@pytest.mark.parametrize("m", [4, 300])
def test_linear_e4m3_keeps_nan_in_its_row(m):
    x, xs, w, ws, _, _ = _linear8(m, 64, 136, 1, False, False)
    clean = la.linear_e4m3(x, xs, w, ws)
    x = x.clone()
    x.view(torch.uint8)[1, 5] = 0x7f   # the NaN of e4m3
    xs = xs.clone()
    xs[2] = float("inf")
    got = la.linear_e4m3(x, xs, w, ws)
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[2]).any()
    others = [i for i in range(m) if i not in (1, 2)]
    assert torch.equal(got[others], clean[others])


# ------------------------------------------------------------------ all of them

def test_no_backward_and_versions():
    x = _inputs(1, 5, 1, 1, 64, 64, F32, seed=1)
    q = x["q"].clone().requires_grad_()
    out, state = la.gated_delta(q, x["k"], x["v"], x["dt"], x["a"], x["beta"], return_state=True)
    with pytest.raises(RuntimeError, match="gated_delta has no backward"):
        out.sum().backward()
    with pytest.raises(RuntimeError, match="gated_delta has no backward"):
        state.sum().backward()
    with pytest.raises(ValueError, match="no gradient passes"):
        la.gated_delta(q, x["k"], x["v"], x["dt"], x["a"], x["beta"], out=torch.empty_like(out))
    w = torch.ones(64, device=DEV, requires_grad=True)
    y, s = la.rms_norm(x["v"][0, :, 0], w, residual=x["k"][0, :, 0])
    with pytest.raises(RuntimeError, match="rms_norm has no backward"):
        y.sum().backward()
    y8, scale = la.rms_norm(x["v"][0, :, 0], w, quantize=True)
    with pytest.raises(RuntimeError, match="rms_norm has no backward"):
        scale.sum().backward()
    held = _randn(_gen(1), 1, 1, 64, 64, scale=0.1)
    before = held._version
    la.gated_delta_step(held, x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], x["dt"][:, 0], x["a"], x["beta"][:, 0])
    assert held._version == before + 1
    with pytest.raises(ValueError, match="updated in place"):
        la.gated_delta_step(held.requires_grad_(), q[:, 0], x["k"][:, 0], x["v"][:, 0], x["dt"][:, 0], x["a"], x["beta"][:, 0])
    with torch.no_grad():
        la.gated_delta_step(held, q[:, 0], x["k"][:, 0], x["v"][:, 0], x["dt"][:, 0], x["a"], x["beta"][:, 0])


def _block(x, w8, ws, w_out8, wos, weight, u):
    """The rule, its gated norm in 8 bits, the projection, and the norm of what follows."""
    out, state = _call(x)
    B, n, hv, dv = out.shape
    gate = u[..., :hv * dv]
    y8, s = la.rms_norm(out.view(B, n, hv * dv), weight, gate=gate, quantize=True)
    r = la.linear_e4m3(y8, s, w8, ws)
    z8, zs, total = la.rms_norm(r, residual=u[..., :r.shape[-1]], quantize=True)
    return la.linear_e4m3(z8, zs, w_out8, wos, residual=total), state, out, y8, s


def test_graphs_and_streams():
    # the run of them captured, replayed with new inputs, and on another stream
    B, n, hk, hv, d = 2, 150, 2, 4, 64
    g = _gen(7)
    w8, ws = _randn(g, 128, hv * d).to(E4M3), torch.rand(128, device=DEV, generator=g) * 0.1
    wo8, wos = _randn(g, 128, 128).to(E4M3), torch.rand(128, device=DEV, generator=g) * 0.1
    weight, u = _randn(g, d, dtype=BF16), _randn(g, B, n, hv * d, dtype=BF16)
    x = _inputs(B, n, hk, hv, d, d, BF16, seed=1)
    fixed = {k: v.clone() for k, v in x.items()}
    want = _block(x, w8, ws, wo8, wos, weight, u)
    graphs, outs = [], []
    for _ in range(2):   # two graphs that may share workspaces
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            outs.append(_block(fixed, w8, ws, wo8, wos, weight, u))
        graphs.append(graph)
    for seed in (2, 1):
        y = _inputs(B, n, hk, hv, d, d, BF16, seed=seed)
        for k in fixed:
            fixed[k].copy_(y[k])
        for graph in graphs:
            graph.replay()
        ref = _block(y, w8, ws, wo8, wos, weight, u)
        for o in outs:
            for a, b in zip(o, ref):
                assert torch.equal(a.float(), b.float())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _block(x, w8, ws, wo8, wos, weight, u)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a.float(), b.float())
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    out = la.gated_delta(x["q"], x["k"], x["v"], x["dt"], x["a"], x["beta"], dt_bias=x["dt_bias"], stream=s2)
    s2.synchronize()
    assert torch.equal(out, want[2])
    assert la.last_device_status() == 0


def test_two_streams_at_once():
    # long enough that both run together; each has its own workspace
    xs = [_inputs(1, 2000, 2, 2, 128, 128, BF16, seed=s) for s in (1, 2)]
    want = [_call(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_call(xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, state in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(state, want[i][1])


def test_block_against_plain():
    # the run as it is used, against 64 bits with the roundings that it makes
    B, n, hk, hv, d = 2, 130, 1, 2, 64
    g = _gen(7)
    w8, ws = _randn(g, 128, hv * d).to(E4M3), torch.rand(128, device=DEV, generator=g) * 0.1
    wo8, wos = _randn(g, 128, 128).to(E4M3), torch.rand(128, device=DEV, generator=g) * 0.1
    weight, u = _randn(g, d, dtype=BF16), _randn(g, B, n, hv * d, dtype=BF16)
    x = _inputs(B, n, hk, hv, d, d, BF16, seed=1)
    got, state, out, y8, s = _block(x, w8, ws, wo8, wos, weight, u)
    _check((out, state), x)
    _norm_close((y8, s), out.view(B, n, hv * d), weight, d, 1e-6, u, None, True)
    r = la.linear_e4m3(y8, s, w8, ws)
    _linear8_close(r.flatten(0, 1), y8.flatten(0, 1), s.flatten(), w8, ws, None, None)
    z8, zs, total = la.rms_norm(r, residual=u, quantize=True)
    _norm_close((z8, zs, total), r, None, 128, 1e-6, None, u, True)
    _linear8_close(got.flatten(0, 1), z8.flatten(0, 1), zs.flatten(), wo8, wos, None, total.flatten(0, 1))


def test_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_delta_block.py")
    spec = importlib.util.spec_from_file_location("gated_delta_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert math.isfinite(example.run(width=256, batch=3, prompt=70, tokens=3))


def test_debug_build_gives_the_same_bits(tmp_path):
    # the LA_DEBUG library in a child process: no check fails, equal outputs
    code = (
        "import sys, torch, causal_kernelized_linear_gb300 as la\n"
        "g = torch.Generator(device='cuda').manual_seed(5)\n"
        "r = lambda *s: torch.randn(*s, device='cuda', generator=g).bfloat16()\n"
        "out = {}\n"
        "def delta(B, n, hk, hv, dk, dv, f32=False, lens=None):\n"
        "    x = [r(B, n, hk, dk), r(B, n, hk, dk), r(B, n, hv, dv), r(B, n, hv), -torch.rand(hv, device='cuda',"
        " generator=g), r(B, n, hv)]\n"
        "    x = [t.float() for t in x] if f32 else x\n"
        "    lens = None if lens is None else torch.tensor(lens, device='cuda', dtype=torch.int32)\n"
        "    return la.gated_delta(*x, lengths=lens, return_state=True)\n"
        "for i, c in enumerate(((1, 200, 1, 2, 128, 136), (2, 77, 1, 1, 64, 40, False, [77, 30]), (1, 2500, 1, 1, 128, 128),"
        " (1, 300, 1, 1, 64, 64, True), (1, 9, 2, 2, 128, 128))):\n"
        "    out[f'delta{i}'], out[f'state{i}'] = delta(*c)\n"
        "for m, k, n in ((5, 208, 136), (130, 528, 1000), (1500, 272, 2056)):\n"
        "    y, s = la.rms_norm(r(m, k), r(k), quantize=True)\n"
        "    w = r(n, k).to(torch.float8_e4m3fn)\n"
        "    out[f'norm{m}'], out[f'scale{m}'] = y.float(), s\n"
        "    out[f'linear{m}'] = la.linear_e4m3(y, s, w, torch.rand(n, device='cuda', generator=g), bias=r(n),"
        " activation='silu', residual=r(m, n))\n"
        "out['status'] = torch.tensor(la.last_device_check())\n"
        "out['debug'] = torch.tensor(int(la.debug_build()))\n"
        "torch.save({k: v.cpu() for k, v in out.items()}, sys.argv[1])\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    la.build()
    la.build(debug=True)
    got = []
    for debug in ("0", "1"):
        path = str(tmp_path / debug)
        env = dict(os.environ, LA_DEBUG=debug, PYTHONPATH=root)
        p = subprocess.run([sys.executable, "-c", code, path], env=env, capture_output=True, text=True, timeout=300)
        assert p.returncode == 0, p.stderr[-2000:]
        got.append(torch.load(path))
    rel, dbg = got
    assert rel.pop("debug").item() == 0 and dbg.pop("debug").item() == 1
    assert rel["status"].tolist() == [0, 0]
    for k in rel:
        assert torch.equal(rel[k], dbg[k]), k


def test_far_offsets():
    # elements past 2^31 in a view, and a batch of states past 2^32 bytes
    n, hv, d = 40, 1, 64
    big = torch.empty(2, n, (1 << 25) + 512, device=DEV, dtype=BF16)   # rows 67 MB apart
    x = _inputs(2, n, 1, hv, d, d, BF16, seed=1)
    y = dict(x)
    for i, name in enumerate(("q", "k", "v")):
        view = big[..., (1 << 25) + i * 64:][..., :64].unflatten(-1, (1, 64))
        view.copy_(x[name])
        y[name] = view
    a, b = _call(x), _call(y)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    del big, y, view
    B, H = 2100, 32
    state = torch.zeros(B, H, 128, 128, device=DEV)
    x = _inputs(B, 1, 1, H, 128, 128, BF16, seed=1)
    s = {k: (v[:, 0] if v.dim() > 1 else v) for k, v in x.items()}
    out = la.gated_delta_step(state, s["q"], s["k"], s["v"], s["dt"], s["a"], s["beta"], dt_bias=s["dt_bias"])
    tail = {k: (v[-3:] if v.dim() > 1 else v) for k, v in x.items()}
    _check((out[-3:, None], state[-3:]), tail, how=TOKENS)
