"""State-space block operators on the GPU against plain 64-bit forms.

Tolerances.  With u = eps/2 of a type (bf16 2^-8, fp32 2^-24), every value may
be off by
* its own rounding: u·|value| for the output's type, and
* the fp32 evaluation of sums: each of the N terms and partial sums of a dot
  product contributes at most 2^-24·Σ|terms|; rounding errors of both signs
  add up to far less than N of them, and 2·sqrt(N) + 16 of them is what the
  tests allow (the 16 covers activations: 2^x, 1/x and their arguments).
The bound is taken element by element from the 64-bit absolute sums.
"""
import math

import pytest
import torch

import causal_kernelized_linear_gb300 as la

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DTYPES = [torch.bfloat16, torch.float32]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, device=DEV, generator=g) * scale).to(dtype)


def _close(got, ref, absum, terms, dtype, what=""):
    """|got − ref| ≤ u·|ref| + (2·sqrt(terms) + 16)·2^-24·absum, element by element."""
    tol = U[dtype] * ref.abs() + (2 * math.sqrt(terms) + 16) * 2.0 ** -24 * absum + 1e-30
    bad = (got.double() - ref).abs() - tol
    worst = bad.max().item() if bad.numel() else 0.0
    assert torch.isfinite(got).all(), what
    assert worst <= 0, f"{what}: off by {worst:.3e} more than allowed"


ACTS = {
    "none": lambda v: v,
    "relu": torch.relu,
    "silu": lambda v: v * torch.sigmoid(v),
    "gelu": lambda v: v * torch.special.ndtr(v),
    "softplus": lambda v: torch.logaddexp(v, torch.zeros_like(v)),
}


# ------------------------------------------------------------------ linear

def _linear_ref(x, w, bias, act, residual):
    xd, wd = x.double(), w.double()
    y = xd @ wd.t()
    ab = xd.abs() @ wd.abs().t()
    if bias is not None:
        y, ab = y + bias.double(), ab + bias.double().abs()
    # |act'| ≤ 1.13 for every activation here, and act's own evaluation is
    # relative to a magnitude of at most |y| + 1
    y, ab = ACTS[act](y), 1.13 * ab + 1.0
    if residual is not None:
        y, ab = y + residual.double(), ab + residual.double().abs()
    return y, ab


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("m,k,n", [
    (1, 8, 8), (1, 4096, 264), (2, 64, 8), (7, 72, 136), (16, 2048, 520), (33, 200, 1000),
    (64, 128, 128), (65, 64, 72), (127, 96, 256), (128, 512, 384), (129, 520, 264),
    (255, 64, 2048), (256, 256, 256), (257, 1032, 520), (700, 40, 8), (1000, 8, 1032),
    (2049, 136, 264), (5000, 72, 640)])
def test_linear_shapes(dtype, m, k, n):
    g = _gen(m * 7 + k * 3 + n)
    x = _randn(g, m, k, dtype=dtype)
    w = _randn(g, n, k, dtype=dtype, scale=k ** -0.5)
    bias = _randn(g, n, dtype=dtype)
    res = _randn(g, m, n, dtype=dtype)
    y = la.linear(x, w, bias=bias, residual=res)
    ref, ab = _linear_ref(x, w, bias, "none", res)
    _close(y, ref, ab, k + 2, dtype)
    assert torch.equal(y, la.linear(x, w, bias=bias, residual=res))   # a fixed order of sums


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("m", [3, 40, 300])
@pytest.mark.parametrize("use_bias,use_res", [(False, False), (True, False), (False, True)])
def test_linear_epilogues(dtype, act, m, use_bias, use_res):
    g = _gen(m)
    k, n = 160, 328
    x = _randn(g, m, k, dtype=dtype, scale=2.0)
    w = _randn(g, n, k, dtype=dtype, scale=k ** -0.5)
    bias = _randn(g, n, dtype=dtype, scale=3.0) if use_bias else None
    res = _randn(g, m, n, dtype=dtype) if use_res else None
    y = la.linear(x, w, bias=bias, activation=act, residual=res)
    ref, ab = _linear_ref(x, w, bias, act, res)
    _close(y, ref, ab, k + 2, dtype, act)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("m", [1, 5, 200, 1025])
def test_linear_views(dtype, m):
    # slices of wider buffers on every side, the residual updated in place,
    # and what lies around the output left alone
    g = _gen(m)
    k, n = 72, 136
    x = _randn(g, m, k + 24, dtype=dtype)[:, 16:16 + k]
    w = _randn(g, n + 3, k + 8, dtype=dtype)[2:2 + n, 8:]
    big = _randn(g, m, n + 48, dtype=dtype)
    keep = big.clone()
    out = big[:, 16:16 + n]
    ref, ab = _linear_ref(x, w, None, "relu", out)
    got = la.linear(x, w, activation="relu", residual=out, out=out)
    assert got.data_ptr() == out.data_ptr()
    _close(got, ref, ab, k + 2, dtype)
    assert torch.equal(big[:, :16], keep[:, :16]) and torch.equal(big[:, 16 + n:], keep[:, 16 + n:])


def test_linear_leading_axes_and_empty():
    g = _gen(3)
    x = _randn(g, 2, 5, 3, 64, dtype=torch.bfloat16)
    w = _randn(g, 72, 64, dtype=torch.bfloat16)
    y = la.linear(x, w)
    assert y.shape == (2, 5, 3, 72)
    assert torch.equal(y.view(-1, 72), la.linear(x.view(-1, 64), w))
    assert la.linear(x[:0], w).shape == (0, 5, 3, 72)
    assert la.linear(x.view(-1, 64)[:0], w).shape == (0, 72)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("m", [4, 300])
def test_linear_keeps_infinities_and_nan_in_their_rows(dtype, m):
    g = _gen(9)
    x = _randn(g, m, 64, dtype=dtype)
    w = _randn(g, 136, 64, dtype=dtype)
    clean = la.linear(x, w)
    x2 = x.clone()
    x2[1, 5] = float("nan")
    x2[2, 7] = float("inf")
    y = la.linear(x2, w)
    assert torch.isnan(y[1]).all()
    assert not torch.isfinite(y[2]).any()
    rest = [i for i in range(m) if i not in (1, 2)]
    assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "softplus"])
def test_linear_activation_extremes(act):
    # products that land on large values of both signs, on zero and on NaN
    vals = torch.tensor([0.0, 1e-6, -1e-6, 30.0, -30.0, 1e4, -1e4, 3e30, -3e30, float("nan")],
                        device=DEV)
    x = torch.zeros(16, 8, device=DEV)
    x[:10, 0] = vals
    w = torch.zeros(8, 8, device=DEV)
    w[0, 0] = 1.0
    y = la.linear(x, w, activation=act)[:10, 0]
    ref = ACTS[act](vals.double())
    if act == "silu":
        ref = torch.where(vals < -1e3, torch.zeros_like(ref), ref)
    assert torch.isnan(y[-1])
    torch.testing.assert_close(y[:-1].double(), ref[:-1], rtol=2e-6, atol=1e-12)


# ------------------------------------------------------------------ convolution

def _conv_ref(x, w, bias, act, state, lens):
    B, n, D = x.shape
    W = w.shape[1]
    past = state if state is not None else x.new_zeros(B, W - 1, D)
    y = torch.zeros(B, n, D, device=x.device, dtype=torch.float64)
    ab = torch.zeros_like(y)
    after = []
    for b in range(B):
        full = torch.cat([past[b], x[b, :lens[b]]]).double()
        o = torch.zeros(lens[b], D, device=x.device, dtype=torch.float64)
        s = torch.zeros_like(o)
        if bias is not None:
            o, s = o + bias.double(), s + bias.double().abs()
        for j in range(W):
            o = o + full[j:j + lens[b]] * w[:, j].double()
            s = s + (full[j:j + lens[b]] * w[:, j].double()).abs()
        y[b, :lens[b]], ab[b, :lens[b]] = ACTS[act](o), 1.13 * s
        after.append(full[lens[b]:])
    return y, ab, torch.stack(after)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,n,D", [(1, 1, 8), (2, 2, 72), (1, 3, 1000), (3, 31, 64), (2, 33, 136),
                                   (1, 257, 520), (5, 130, 8), (1, 2000, 64)])
@pytest.mark.parametrize("act,use_bias,use_state", [("silu", True, False), ("none", False, True)])
def test_conv_shapes(dtype, W, B, n, D, act, use_bias, use_state):
    g = _gen(B + n + D + W)
    x = _randn(g, B, n, D, dtype=dtype)
    w = _randn(g, D, W, dtype=dtype)
    bias = _randn(g, D, dtype=dtype) if use_bias else None
    st = _randn(g, B, W - 1, D, dtype=dtype) if use_state else None
    y, after = la.causal_conv(x, w, bias=bias, activation=act, state=st, return_state=True)
    ref, ab, ref_after = _conv_ref(x, w, bias, act, st, [n] * B)
    _close(y, ref, ab, W + 1, dtype)
    assert torch.equal(after.double(), ref_after)
    assert torch.equal(y, la.causal_conv(x, w, bias=bias, activation=act, state=st))


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_lengths(dtype, W):
    # lengths of 0, 1, shorter than the width, across a run's border, the
    # whole, and out of range both ways; what lies past a length is NaN
    n, D = 70, 72
    lens = [0, 1, 2, 32, 33, 63, 64, 70, -5, 1000]
    eff = [min(max(v, 0), n) for v in lens]
    g = _gen(W)
    B = len(lens)
    x = _randn(g, B, n, D, dtype=dtype)
    w, bias = _randn(g, D, W, dtype=dtype), _randn(g, D, dtype=dtype)
    st = _randn(g, B, W - 1, D, dtype=dtype)
    ref, ab, ref_after = _conv_ref(x, w, bias, "silu", st, eff)
    for b, v in enumerate(eff):
        x[b, v:] = float("nan")
    y, after = la.causal_conv(x, w, bias=bias, state=st, return_state=True,
                              lengths=torch.tensor(lens, device=DEV, dtype=torch.int32))
    _close(y, ref, ab, W + 1, dtype)
    for b, v in enumerate(eff):
        assert (y[b, v:] == 0).all()
    assert torch.equal(after.double(), ref_after)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_conv_views_and_empty(dtype):
    g = _gen(4)
    big = _randn(g, 3, 50, 200, dtype=dtype)
    w = _randn(g, 64, 4, dtype=dtype)
    x = big[..., 72:136]
    y = la.causal_conv(x, w)
    assert torch.equal(y, la.causal_conv(x.contiguous(), w))
    # token-major memory, and a slice of a wider buffer as the output
    xt = x.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((3, 50, 96), 7.0, device=DEV, dtype=dtype)
    assert torch.equal(la.causal_conv(xt, w, out=wide[..., 16:80]), y)
    assert (wide[..., :16] == 7).all() and (wide[..., 80:] == 7).all()
    st = _randn(g, 3, 3, 64, dtype=dtype)
    empty, after = la.causal_conv(x[:, :0], w, state=st, return_state=True)
    assert empty.shape == (3, 0, 64) and torch.equal(after, st)
    _, after = la.causal_conv(x[:, :0], w, return_state=True)
    assert (after == 0).all()
    assert la.causal_conv(x[:0], w).shape == (0, 50, 64)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_conv_steps_follow_the_prompt(dtype, W, act):
    # a prompt in one call = its first part, then token by token, bit for bit
    g = _gen(W)
    B, n, D = 3, 12, 72
    x = _randn(g, B, n, D, dtype=dtype)
    w, bias = _randn(g, D, W, dtype=dtype), _randn(g, D, dtype=dtype)
    whole, end = la.causal_conv(x, w, bias=bias, activation=act, return_state=True)
    _, state = la.causal_conv(x[:, :5], w, bias=bias, activation=act, return_state=True)
    for t in range(5, n):
        y = la.causal_conv_step(state, x[:, t], w, bias=bias, activation=act)
        assert torch.equal(y, whole[:, t]), t
    assert torch.equal(state, end)
    xi = x[:, 0].clone()
    s1, s2 = end.clone(), end.clone()
    y = la.causal_conv_step(s1, xi.clone(), w, activation=act)
    assert torch.equal(la.causal_conv_step(s2, xi, w, activation=act, out=xi), y)   # in place


# ------------------------------------------------------------------ scan

def _scan_inputs(g, B, n, D, S, dtype, gate=True, state=False, scale_dt=0.5):
    i = {"x": _randn(g, B, n, D, dtype=dtype), "dt": _randn(g, B, n, D, dtype=dtype, scale=scale_dt),
         "a": -torch.rand(D, S, device=DEV, generator=g) * S,
         "b": _randn(g, B, n, S, dtype=dtype), "c": _randn(g, B, n, S, dtype=dtype),
         "skip": _randn(g, D, dtype=torch.float32),
         "dt_bias": _randn(g, D, dtype=torch.float32) - 3.0,
         "gate": _randn(g, B, n, D, dtype=dtype) if gate else None,
         "state": _randn(g, B, D, S, dtype=torch.float32) if state else None}
    return i


def _scan_ref(i, lens=None, softplus=True):
    """(y, its absolute sums, h, its absolute sums) in 64 bits, token by token.
    The absolute sum of the state runs with the same decays and takes in, for
    every step, the relative error of that step's decay: its argument's
    rounding (|Δ·a| ulps) beside the step's own."""
    f = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in i.items()}
    B, n, D = f["x"].shape
    S = f["a"].shape[1]
    dt = f["dt"] + (f["dt_bias"] if f["dt_bias"] is not None else 0.0)
    dt = ACTS["softplus"](dt) if softplus else dt
    h = f["state"].clone() if f["state"] is not None else torch.zeros(B, D, S, device=DEV, dtype=torch.float64)
    hs = h.abs()
    y, ys = torch.zeros_like(f["x"]), torch.zeros_like(f["x"])
    for t in range(n):
        live = torch.ones(B, 1, 1, device=DEV, dtype=torch.bool) if lens is None else \
            (t < torch.tensor(lens, device=DEV))[:, None, None]
        arg = dt[:, t, :, None] * f["a"]
        u = (dt[:, t] * f["x"][:, t])[..., None] * f["b"][:, t, None]
        h = torch.where(live, torch.exp(arg) * h + u, h)
        hs = torch.where(live, torch.exp(arg) * hs + u.abs(), hs)
        y[:, t] = (h * f["c"][:, t, None]).sum(-1)
        ys[:, t] = (hs * f["c"][:, t, None].abs()).sum(-1)
    if f["skip"] is not None:
        y, ys = y + f["skip"] * f["x"], ys + (f["skip"] * f["x"]).abs()
    if f["gate"] is not None:
        z = ACTS["silu"](f["gate"])
        y, ys = y * z, ys * z.abs()
    if lens is not None:
        dead = torch.arange(n, device=DEV)[None] >= torch.tensor(lens, device=DEV)[:, None]
        y[dead], ys[dead] = 0.0, 0.0
    return y, ys, h, hs


def _scan_check(i, got, after, lens=None, softplus=True):
    # Errors of the decays add over the steps a term survives: a term decays by
    # e^{−Σ|Δ·a|}, its relative error is at most (Σ|Δ·a| + 3·steps)·2^-24 before the
    # weight e^{−Σ|Δ·a|}; over random signs sqrt(steps) of them.  The number of
    # terms in _close therefore counts the tokens.
    y, ys, h, hs = _scan_ref(i, lens, softplus)
    n, S = i["x"].shape[1], i["a"].shape[1]
    _close(got, y, 4 * ys, n + S, i["x"].dtype, "y")
    _close(after, h, 4 * hs, n + S, torch.float32, "state")


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("B,n,D", [(1, 1, 8), (2, 2, 72), (3, 5, 64), (1, 33, 1000), (2, 64, 136),
                                   (1, 129, 8), (1, 700, 64), (1, 3001, 8)])
def test_scan_shapes(dtype, S, B, n, D):
    i = _scan_inputs(_gen(B + n + D + S), B, n, D, S, dtype, gate=n % 2 == 1, state=D % 16 == 8)
    got, after = la.selective_scan(**i, return_state=True)
    _scan_check(i, got, after)
    again, end = la.selective_scan(**i, return_state=True)
    assert torch.equal(got, again) and torch.equal(after, end)
    assert torch.equal(got, la.selective_scan(**i))


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 64])
@pytest.mark.parametrize("n", [70, 900])
def test_scan_lengths(dtype, S, n):
    lens = [0, 1, 3, 31, 32, 33, 64, n, -1, 5000, n - 1, n // 2]
    eff = [min(max(v, 0), n) for v in lens]
    i = _scan_inputs(_gen(S), len(lens), n, 40, S, dtype, state=True)
    y, ys, h, hs = _scan_ref(i, eff)
    for k in ("x", "dt", "b", "c", "gate"):
        for b, v in enumerate(eff):
            i[k][b, v:] = float("nan") if b % 2 else float("inf")
    got, after = la.selective_scan(**i, return_state=True,
                                   lengths=torch.tensor(lens, device=DEV, dtype=torch.int32))
    _close(got, y, 4 * ys, n + S, dtype, "y")
    _close(after, h, 4 * hs, n + S, torch.float32, "state")
    for b, v in enumerate(eff):
        assert (got[b, v:] == 0).all()
    assert torch.equal(after[0], i["state"][0])


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_optional_terms(dtype, softplus):
    i = _scan_inputs(_gen(1), 2, 40, 72, 16, dtype, gate=False)
    if not softplus:
        i["dt"] = i["dt"].abs()
    for drop in ((), ("skip",), ("dt_bias",), ("skip", "dt_bias")):
        j = dict(i, **{k: None for k in drop})
        if not softplus:
            j["dt_bias"] = None
        got, after = la.selective_scan(**j, softplus=softplus, return_state=True)
        _scan_check(j, got, after, softplus=softplus)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_scan_extreme_steps(dtype):
    # steps of zero and steps that erase the state, and far-negative raw steps
    i = _scan_inputs(_gen(2), 2, 64, 72, 16, dtype)
    i["dt"][:, ::7] = -80.0
    i["dt"][:, 3::7] = 60.0
    got, after = la.selective_scan(**i, return_state=True)
    _scan_check(i, got, after)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_scan_views_and_empty(dtype):
    g = _gen(6)
    B, n, D, S = 3, 45, 72, 16
    i = _scan_inputs(g, B, n, D, S, dtype)
    want, end = la.selective_scan(**i, return_state=True)
    xz = torch.cat([i["x"], i["gate"]], -1)
    bc = torch.cat([i["x"][..., :8], i["b"], i["c"]], -1)
    j = dict(i, x=xz[..., :D], gate=xz[..., D:], b=bc[..., 8:8 + S], c=bc[..., 8 + S:],
             dt=i["dt"].transpose(0, 1).contiguous().transpose(0, 1))
    wide = torch.full((B, n, D + 32), 7.0, device=DEV, dtype=dtype)
    got, after = la.selective_scan(**j, return_state=True, out=wide[..., 16:16 + D])
    assert torch.equal(got, want) and torch.equal(after, end)
    assert (wide[..., :16] == 7).all() and (wide[..., 16 + D:] == 7).all()
    # b and c shared by the whole batch: a stride of zero
    j = dict(i, b=i["b"][:1].expand(B, n, S), c=i["c"][:1].expand(B, n, S))
    k = dict(i, b=j["b"].contiguous(), c=j["c"].contiguous())
    assert torch.equal(la.selective_scan(**j), la.selective_scan(**k))
    cut = {q: (v[:, :0] if q in ("x", "dt", "b", "c", "gate") else v) for q, v in i.items()}
    empty, after = la.selective_scan(**cut, return_state=True)
    assert empty.shape == (B, 0, D) and (after == 0).all()
    cut["state"] = end
    assert torch.equal(la.selective_scan(**cut, return_state=True)[1], end)


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("B,D", [(1, 8), (2, 72), (5, 1000), (64, 136)])
def test_step(dtype, S, B, D):
    i = _scan_inputs(_gen(S + B), B, 1, D, S, dtype, gate=D != 72, state=True)
    y, ys, h, hs = _scan_ref(i)
    one = {k: (v[:, 0] if k in ("x", "dt", "b", "c", "gate") and v is not None else v)
           for k, v in i.items()}
    st = one.pop("state").clone()
    got = la.selective_step(st, **one)
    _close(got, y[:, 0], 4 * ys[:, 0], S + 1, dtype, "y")
    _close(st, h, 4 * hs, S + 1, torch.float32, "state")


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_steps_follow_the_prompt(dtype):
    i = _scan_inputs(_gen(8), 2, 30, 72, 16, dtype)
    first = {k: (v[:, :20] if k in ("x", "dt", "b", "c", "gate") else v) for k, v in i.items()}
    _, state = la.selective_scan(**first, return_state=True)
    y, ys, h, hs = _scan_ref(i)
    i.pop("state")
    for t in range(20, 30):
        one = {k: (v[:, t] if k in ("x", "dt", "b", "c", "gate") else v) for k, v in i.items()}
        got = la.selective_step(state, **one)
        _close(got, y[:, t], 4 * ys[:, t], 30 + 16, dtype, f"token {t}")
    _close(state, h, 4 * hs, 30 + 16, torch.float32, "state")


# ------------------------------------------------------------------ streams and graphs

def test_streams_and_graph_capture():
    g = _gen(11)
    i = _scan_inputs(g, 1, 600, 64, 16, torch.bfloat16)
    w = _randn(g, 136, 64, dtype=torch.bfloat16, scale=0.1)
    cw = _randn(g, 64, 4, dtype=torch.bfloat16)

    def block(stream=None):
        x = la.causal_conv(i["x"], cw, stream=stream)
        y = la.selective_scan(**dict(i, x=x), stream=stream)
        return la.linear(y, w, activation="silu", stream=stream)

    want = block()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = block(side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    i["x"].copy_(_randn(g, 1, 600, 64, dtype=torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, block())
    assert la.last_device_status() == 0


# ------------------------------------------------------------------ sizes of the larger kernels

@pytest.mark.parametrize("m,k,n", [
    (6000, 64, 2056),      # several waves of 256-column pairs, a ragged last column
    (1024, 520, 2048),     # 128-column pairs, K off 64
    (2500, 1000, 1288), (700, 2048, 2048), (4099, 8, 4096), (300, 4096, 520), (129, 4096, 4096)])
@pytest.mark.parametrize("act,use_bias,use_res", [("none", False, False), ("silu", True, True)])
def test_linear_bf16_kernels(m, k, n, act, use_bias, use_res):
    g = _gen(m + n)
    x = _randn(g, m, k, dtype=torch.bfloat16)
    w = _randn(g, n, k, dtype=torch.bfloat16, scale=k ** -0.5)
    bias = _randn(g, n, dtype=torch.bfloat16) if use_bias else None
    res = _randn(g, m, n, dtype=torch.bfloat16) if use_res else None
    y = la.linear(x, w, bias=bias, activation=act, residual=res)
    ref, ab = _linear_ref(x, w, bias, act, res)
    _close(y, ref, ab, k + 2, torch.bfloat16)
    again = res.clone() if use_res else torch.empty_like(y)
    la.linear(x, w, bias=bias, activation=act, residual=again if use_res else None, out=again)
    assert torch.equal(again, y)
    assert la.last_device_status() == 0


@pytest.mark.parametrize("m,k,n", [
    (9, 36, 20), (100, 2048, 1032), (200, 512, 1024), (400, 1024, 512), (777, 128, 4096),
    (1000, 1028, 1024), (3000, 68, 1000), (64, 4096, 64)])
@pytest.mark.parametrize("act,use_bias,use_res", [("none", False, False), ("gelu", True, True)])
def test_linear_f32_kernels(m, k, n, act, use_bias, use_res):
    g = _gen(m + n)
    x = _randn(g, m, k, dtype=torch.float32)
    w = _randn(g, n, k, dtype=torch.float32, scale=k ** -0.5)
    bias = _randn(g, n, dtype=torch.float32) if use_bias else None
    res = _randn(g, m, n, dtype=torch.float32) if use_res else None
    y = la.linear(x, w, bias=bias, activation=act, residual=res)
    ref, ab = _linear_ref(x, w, bias, act, res)
    _close(y, ref, ab, k + 2, torch.float32)
    assert torch.equal(y, la.linear(x, w, bias=bias, activation=act, residual=res))


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("S", [16, 32])
def test_scan_chunks_and_lengths(dtype, S):
    # a sequence long enough for many chunks; lengths on, before and after a
    # chunk's border, and in its first chunk
    n = 2100
    lens = [n, 0, 64, 65, 1024, 1030, 2090]
    i = _scan_inputs(_gen(S), len(lens), n, 24, S, dtype, state=True)
    y, ys, h, hs = _scan_ref(i, lens)
    got, after = la.selective_scan(**i, return_state=True,
                                   lengths=torch.tensor(lens, device=DEV, dtype=torch.int32))
    _close(got, y, 4 * ys, n + S, dtype, "y")
    _close(after, h, 4 * hs, n + S, torch.float32, "state")


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 64])
@pytest.mark.parametrize("B", [4, 9, 300])
def test_step_batches(dtype, S, B):
    # enough elements for four batch entries per lane, with a remainder
    D = 2048
    i = _scan_inputs(_gen(S + B), B, 1, D, S, dtype, state=True)
    y, ys, h, hs = _scan_ref(i)
    one = {k: (v[:, 0] if k in ("x", "dt", "b", "c", "gate") and v is not None else v)
           for k, v in i.items()}
    st = one.pop("state").clone()
    got = la.selective_step(st, **one)
    _close(got, y[:, 0], 4 * ys[:, 0], S + 1, dtype, "y")
    _close(st, h, 4 * hs, S + 1, torch.float32, "state")


# ------------------------------------------------------------------ offsets past 32 bits

def test_offsets_past_32_bits():
    g = _gen(21)
    far = (1 << 31) + 4096
    big = torch.zeros(far + (1 << 16), device=DEV, dtype=torch.bfloat16)
    D, n = 64, 40

    def spread(t):       # batch entry 1 lies 2^31 elements after entry 0
        v = big.as_strided((2, n, D), (far, D, 1))
        v.copy_(t)
        return v

    x = _randn(g, 2, n, D, dtype=torch.bfloat16)
    w = _randn(g, D, 4, dtype=torch.bfloat16)
    want = la.causal_conv(x, w)
    assert torch.equal(la.causal_conv(spread(x), w), want)
    i = _scan_inputs(g, 2, n, D, 16, torch.bfloat16)
    want, end = la.selective_scan(**i, return_state=True)
    got, after = la.selective_scan(**dict(i, x=spread(i["x"])), return_state=True)
    assert torch.equal(got, want) and torch.equal(after, end)
    out = big.as_strided((2, n, D), (far, D, 1))
    la.selective_scan(**i, out=out)
    assert torch.equal(out, want)
    st = end.clone()
    one = {k: (v[:, 0] if k in ("x", "dt", "b", "c", "gate") else v) for k, v in i.items()}
    one.pop("state")
    y = la.selective_step(st, **one)
    st2 = end.clone()
    xs = spread(i["x"])[:, 0]
    assert torch.equal(la.selective_step(st2, **dict(one, x=xs)), y) and torch.equal(st, st2)
    # rows of x 2^28 elements apart
    del out, xs
    rows = big.as_strided((9, 64), (1 << 28, 1))
    xl = _randn(g, 9, 64, dtype=torch.bfloat16)
    rows.copy_(xl)
    wl = _randn(g, 136, 64, dtype=torch.bfloat16)
    assert torch.equal(la.linear(rows, wl), la.linear(xl, wl))


# ------------------------------------------------------------------ the block as a whole

def test_example_block_prompt_and_tokens_agree():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "state_space_block.py")
    spec = importlib.util.spec_from_file_location("state_space_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    # every value passes through eight bf16 roundings on either path (2^-8 each,
    # relative to values that the residual keeps near the largest): 2^-5
    assert mod.run(width=128, batch=3, prompt=70, tokens=5) <= 2.0 ** -5
    assert mod.run(width=512, batch=2, prompt=300, tokens=3) <= 2.0 ** -5


def test_debug_build_gives_the_same_bits():
    # the LA_DEBUG library in a child process: no check fails, equal outputs
    import subprocess
    import sys
    import tempfile
    code = (
        "import sys, torch, causal_kernelized_linear_gb300 as la\n"
        "g = torch.Generator(device='cuda').manual_seed(5)\n"
        "r = lambda *s: torch.randn(*s, device='cuda', generator=g).bfloat16()\n"
        "out = {}\n"
        "for m, k, n in ((5, 200, 136), (130, 520, 1000), (3000, 264, 2056)):\n"
        "    out[f'{m}'] = la.linear(r(m, k), r(n, k), bias=r(n), activation='silu', residual=r(m, n))\n"
        "out['conv'] = la.causal_conv(r(2, 77, 72), r(72, 4))\n"
        "out['scan'] = la.selective_scan(r(1, 700, 72), r(1, 700, 72), -torch.rand(72, 16,"
        " device='cuda', generator=g), r(1, 700, 16), r(1, 700, 16))\n"
        "out['status'] = torch.tensor(la.last_device_check())\n"
        "out['debug'] = torch.tensor(int(la.debug_build()))\n"
        "torch.save({k: v.cpu() for k, v in out.items()}, sys.argv[1])\n")
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    la.build()
    la.build(debug=True)
    got = []
    with tempfile.TemporaryDirectory() as d:
        for debug in ("0", "1"):
            path = os.path.join(d, debug)
            env = dict(os.environ, LA_DEBUG=debug, PYTHONPATH=root)
            p = subprocess.run([sys.executable, "-c", code, path], env=env, capture_output=True,
                               text=True, timeout=300)
            assert p.returncode == 0, p.stderr[-2000:]
            got.append(torch.load(path))
    rel, dbg = got
    assert rel.pop("debug").item() == 0 and dbg.pop("debug").item() == 1
    assert rel["status"].tolist() == [0, 0]
    for k in rel:
        assert torch.equal(rel[k], dbg[k]), k


@pytest.mark.parametrize("dtype", DTYPES, ids=["bf16", "f32"])
def test_conv_long_runs(dtype):
    # enough channels for runs of 64 tokens; lengths inside, at and past a run's border
    n, D, W = 1300, 4096, 4
    lens = [n, 0, 1, 63, 64, 65, 1279, 1280]
    g = _gen(31)
    x = _randn(g, len(lens), n, D, dtype=dtype)
    w, bias = _randn(g, D, W, dtype=dtype), _randn(g, D, dtype=dtype)
    st = _randn(g, len(lens), W - 1, D, dtype=dtype)
    ref, ab, ref_after = _conv_ref(x, w, bias, "silu", st, lens)
    y, after = la.causal_conv(x, w, bias=bias, state=st, return_state=True,
                              lengths=torch.tensor(lens, device=DEV, dtype=torch.int32))
    _close(y, ref, ab, W + 1, dtype)
    assert torch.equal(after.double(), ref_after)


@pytest.mark.parametrize("n", [50, 700])
def test_scan_rates_of_minus_infinity_and_lengths(n):
    # exp(Δ·(−inf)) = 0: such a state holds the newest token only; tokens past
    # the length still leave it alone
    lens = [n, 0, 1, n - 7]
    i = _scan_inputs(_gen(41), len(lens), n, 24, 16, torch.float32, state=True)
    i["a"][:, 3] = float("-inf")
    y, ys, h, hs = _scan_ref(i, lens)
    got, after = la.selective_scan(**i, return_state=True,
                                   lengths=torch.tensor(lens, device=DEV, dtype=torch.int32))
    _close(got, y, 4 * ys, n + 16, torch.float32, "y")
    _close(after, h, 4 * hs, n + 16, torch.float32, "state")


def test_refusals_queue_nothing():
    g = _gen(51)
    bf = torch.bfloat16
    x, w = _randn(g, 4, 64, dtype=bf), _randn(g, 32, 64, dtype=bf)
    seq = _randn(g, 2, 10, 64, dtype=bf)
    cw = _randn(g, 64, 4, dtype=bf)
    i = _scan_inputs(g, 2, 10, 64, 16, bf)
    la.linear(x, w)
    before = la.launch_count()
    refused = [
        lambda: la.linear(x, w[:, :56]),                                  # K differs
        lambda: la.linear(_randn(g, 4, 72, dtype=bf)[:, 1:65], w),        # not 16-byte aligned
        lambda: la.linear(_randn(g, 4, 68, dtype=bf)[:, :64], w),         # row stride off 16 bytes
        lambda: la.linear(x[:, :60], w[:, :60]),                          # K off 16 bytes
        lambda: la.linear(x[:1].expand(4, 64), w),                        # rows coincide
        lambda: la.causal_conv(seq, _randn(g, 64, 5, dtype=bf)),          # five taps
        lambda: la.causal_conv(seq, cw, activation="gelu"),
        lambda: la.selective_scan(**dict(i, b=i["b"][..., :8], c=i["c"][..., :8])),
        lambda: la.selective_scan(**dict(i, out=i["x"][:, :1].expand(2, 10, 64))),
    ]
    for f in refused:
        with pytest.raises(la.LinAttnError):
            f()
    wrong = [
        lambda: la.linear(x, w.float()),
        lambda: la.linear(x.t(), w),
        lambda: la.linear(x, w, bias=_randn(g, 31, dtype=bf)),
        lambda: la.linear(x, w, residual=_randn(g, 4, 24, dtype=bf)),
        lambda: la.linear(x, w, out=torch.empty(4, 24, device=DEV, dtype=bf)),
        lambda: la.linear(x, w, activation="swish"),
        lambda: la.linear(x, w.cpu()),
        lambda: la.causal_conv(seq, cw, lengths=torch.zeros(2, device=DEV, dtype=torch.int64)),
        lambda: la.causal_conv(seq, cw, lengths=torch.zeros(3, device=DEV, dtype=torch.int32)),
        lambda: la.causal_conv(seq, cw, state=torch.zeros(2, 4, 64, device=DEV, dtype=bf)),
        lambda: la.causal_conv(seq[0], cw),
        lambda: la.selective_scan(**dict(i, a=i["a"].t())),
        lambda: la.selective_scan(**dict(i, a=i["a"].to(bf))),
        lambda: la.selective_scan(**dict(i, state=torch.zeros(2, 64, 8, device=DEV))),
        lambda: la.selective_scan(**dict(i, gate=i["gate"].float())),
    ]
    for f in wrong:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        la.selective_step(None, *[i[k][:, 0] for k in ("x", "dt")], i["a"], i["b"][:, 0], i["c"][:, 0])
    assert la.launch_count() == before and la.last_device_status() == 0
