"""State-space block operators on the GPU: order with the kernels before them,
accuracy where a value is small, aliases, gradients and the sizes at which
another kernel takes over."""
import ctypes
import math

import pytest
import torch

import causal_kernelized_linear_gb300 as la
from test_block_gpu import _close, _linear_ref, _scan_inputs, _scan_ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, device=DEV, generator=g) * scale).to(dtype)


# ------------------------------------------------------------------ order with the kernel before

class _Dim3(ctypes.Structure):
    _fields_ = [("x", ctypes.c_uint), ("y", ctypes.c_uint), ("z", ctypes.c_uint)]


class _KernelParams(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", _Dim3), ("block", _Dim3), ("smem", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p)]


def _second_launch(f):
    """(starts early, CTAs, dynamic shared memory) of the second of f's two kernels, from
    the graph that they record."""
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        f()
    rt = la.load()                               # the CUDA runtime that the library is linked to
    rt.cudaGraphGetEdges.argtypes = [ctypes.c_void_p] * 5
    rt.cudaGraphKernelNodeGetParams.argtypes = [ctypes.c_void_p] * 2
    n = ctypes.c_size_t()
    raw = graph.raw_cuda_graph()
    assert rt.cudaGraphGetEdges(raw, None, None, None, ctypes.byref(n)) == 0 and n.value == 1
    ends = [(ctypes.c_void_p * 1)() for _ in range(2)]
    data = (ctypes.c_uint8 * 8)()                # from_port, to_port, type, reserved
    assert rt.cudaGraphGetEdges(raw, ends[0], ends[1], data, ctypes.byref(n)) == 0
    p = _KernelParams()
    assert rt.cudaGraphKernelNodeGetParams(ends[1][0], ctypes.byref(p)) == 0
    return data[2] == 1, p.grid.x * p.grid.y * p.grid.z, p.smem


def _spread_evenly(launch):
    """In its predecessor's tail a grid that fits on the GPU at once would crowd the SMs
    that have room first: it waits, or an SM does not take more than its share of it
    (228 KB of shared memory, 1 KB of them per CTA)."""
    early, ctas, smem = launch
    share = -(-ctas // torch.cuda.get_device_properties(0).multi_processor_count)
    return not early or (share + 1) * (smem + 1024) > 228 * 1024


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,n,D,S", [(1, 100, 64, 16), (4, 500, 2048, 16), (8, 130, 2048, 8), (5, 400, 1024, 32),
                                     (3, 200, 2048, 64)])
def test_scan_is_spread_evenly_in_its_predecessors_tail(dtype, B, n, D, S):
    g = _gen(1)
    x, dt = (_randn(g, B, n, D, dtype=dtype) for _ in range(2))
    b, c = _randn(g, B, n, S, dtype=dtype), _randn(g, B, n, S, dtype=dtype)
    a = -torch.rand(D, S, device=DEV, generator=g)
    cw = _randn(g, D, 4, dtype=dtype)
    out, y = torch.empty_like(x), torch.empty_like(x)

    def conv_scan():
        la.causal_conv(x, cw, out=y)
        la.selective_scan(y, dt, a, b, c, out=out)
    assert _spread_evenly(_second_launch(conv_scan))


@pytest.mark.parametrize("m,k,n", [(400, 1024, 512), (24, 80, 4096), (200, 512, 1024), (777, 256, 2048),
                                   (723, 236, 1076), (97, 2044, 1404)])
def test_fp32_tiles_are_spread_evenly_in_their_predecessors_tail(m, k, n):
    g = _gen(2)
    f32 = torch.float32
    assert la.selftest_linear_kernel(f32, m, n, k).startswith("tile")
    x, w, cw = _randn(g, m, k, dtype=f32), _randn(g, n, k, dtype=f32, scale=0.1), _randn(g, k, 4, dtype=f32)
    out, y = torch.empty(m, n, device=DEV), torch.empty(1, m, k, device=DEV)

    def conv_linear():
        la.causal_conv(x[None], cw, out=y)
        la.linear(y[0], w, out=out)
    assert _spread_evenly(_second_launch(conv_linear))


def test_products_between_the_attention_kernels():
    """The attention's tensor-core kernels, which take a whole SM's tensor memory
    and start their own followers early, before, after and beside the products,
    on one stream and on two: the same bits as one call at a time."""
    g = _gen(3)
    B, H, n, d = 1, 8, 1024, 64
    x = _randn(g, B * H * n, 64)
    w = [_randn(g, 64, 64, scale=0.125) for _ in range(3)]
    few = _randn(g, 40, 512)
    wf = _randn(g, 512, 512, scale=512 ** -0.5)
    decay = torch.full((H,), 0.98, device=DEV)

    def attend():
        q, k, v = (la.linear(x, m).view(B, H, n, d) for m in w)
        la.forward_state(k, v, decay)
        y = la.linear(few, wf, activation="silu")
        o = la.forward(q, k, v, decay)
        la.forward_state(q, o, decay)
        z = la.linear(y, wf, residual=few)
        return la.linear(o.view(-1, d), w[0], residual=x), z

    want = []
    q, k, v = (la.linear(x, m).view(B, H, n, d) for m in w)
    torch.cuda.synchronize()
    o = la.forward(q, k, v, decay)
    torch.cuda.synchronize()
    y = la.linear(few, wf, activation="silu")
    torch.cuda.synchronize()
    want = la.linear(o.view(-1, d), w[0], residual=x), la.linear(y, wf, residual=few)
    torch.cuda.synchronize()
    for _ in range(3):
        got = attend()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = attend()
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(p, q) for p, q in zip(pair, want))
    assert la.last_device_status() == 0


# ------------------------------------------------------------------ rates of minus infinity

@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,D,S", [(2, 72, 16), (300, 2048, 8)])
def test_step_with_rates_of_minus_infinity(dtype, B, D, S):
    """exp(Δ·(−inf)) is 0 for Δ > 0, and a step of zero leaves the state alone, as
    in the scan: the next token's step after the prompt's gives the same state."""
    g = _gen(4)
    a = -torch.rand(D, S, device=DEV, generator=g)
    a[:, 3] = -math.inf
    state = torch.randn(B, D, S, device=DEV, generator=g)
    x, b, c = _randn(g, B, D, dtype=dtype), _randn(g, B, S, dtype=dtype), _randn(g, B, S, dtype=dtype)
    dt = _randn(g, B, D, dtype=dtype).abs()
    dt[:, ::3] = 0.0
    st = state.clone()
    y = la.selective_step(st, x, dt, a, b, c, softplus=False)
    want = torch.where(dt.double()[..., None] > 0, torch.exp(dt.double()[..., None] * a), 1.0) * state \
        + (dt.double() * x)[..., None] * b[:, None]
    assert torch.isfinite(st).all() and torch.isfinite(y).all()
    assert torch.equal(st[:, ::3], state[:, ::3])
    # the decay's 2^x and argument: a few ulp of 2^-24 of the largest term, far below 1e-5
    assert ((st - want).abs() <= 1e-5 * (want.abs() + state.abs() + 1)).all()
    scan, end = la.selective_scan(x[:, None], dt[:, None], a, b[:, None], c[:, None], softplus=False,
                                  state=state, return_state=True)
    assert ((end - st).abs() <= 1e-5 * (st.abs() + state.abs() + 1)).all()


# ------------------------------------------------------------------ activations where they are small

def _through_linear(v, act, rows, dtype):
    """act of the values v, each the only term of its product, in calls of `rows` rows."""
    v = v.to(dtype)
    w = torch.eye(64, device=DEV, dtype=dtype)
    y = torch.empty_like(v)
    for i in range(0, v.numel(), rows * 64):
        y[i:i + rows * 64] = la.linear(v[i:i + rows * 64].view(-1, 64), w, activation=act).view(-1)
    return v.double(), y.double()


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [2, 8, 64, 1024])
def test_gelu_relative_accuracy(dtype, rows):
    """x·Φ(x) where Φ is small.  Φ(−u) has e^{−u²/2}: the square, its product with
    log2(e)/2 and that constant round by 2^-24 each at most, which the
    exponential turns into 1.5·x²·2^-24 relative below zero; 2^x, 1/x, a fitted
    polynomial and four products stay within 20·2^-24.  Beside it the output's
    own rounding.  Above zero Φ's small error is relative to 1 − Φ(−x) ≥ 1/2."""
    x, y = _through_linear(torch.linspace(-12, 12, 64 * 2048, device=DEV), "gelu", rows, dtype)
    ref = 0.5 * x * torch.special.erfc(-x * math.sqrt(0.5))
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    tol = (half + (1.5 * x.clamp(max=0) ** 2 + 20) * 2.0 ** -24) * ref.abs()
    assert ((y - ref).abs() <= tol).all(), ((y - ref).abs() / ref.abs().clamp_min(1e-300)).max()
    far = torch.tensor([-1e4, -60.0, -15.0, 0.0, 60.0, 1e4, -1e30, 1e30] * 16, device=DEV)
    x, y = _through_linear(far, "gelu", rows, dtype)
    assert (y[x <= 0].abs() <= 1e-30).all() and torch.equal(y[x > 0], x[x > 0])


def _silu(x):
    return x * torch.sigmoid(x)


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _relative(x, y, ref, dtype, fixed):
    """e^{−|x|} comes from an exponent that rounds by 2^-24 of itself and a constant off by
    a quarter of that: 1.25·|x|·2^-24 relative where it decides the value, below zero;
    `fixed` roundings of 2^-24 (2^x counts four, 1/x two) beside it, and the output's."""
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    tol = (half + (1.25 * (-x).clamp(min=0) + fixed) * 2.0 ** -24) * ref.abs()
    worst = ((y - ref).abs() - tol).max()
    assert ((y - ref).abs() <= tol).all(), worst


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [2, 8, 64, 1024])
@pytest.mark.parametrize("act,ref,fixed", [("silu", _silu, 9), ("softplus", _softplus, 12)])
def test_relative_accuracy_through_linear(dtype, rows, act, ref, fixed):
    x, y = _through_linear(torch.linspace(-80, 80, 64 * 2048, device=DEV), act, rows, dtype)
    _relative(x, y, ref(x), dtype, fixed)


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
def test_relative_accuracy_of_the_convolution_and_the_gate(dtype):
    v = torch.linspace(-80, 80, 64 * 2048, device=DEV).to(dtype)
    x = v.view(1, -1, 64)
    w = torch.zeros(64, 2, device=DEV, dtype=dtype)
    w[:, 1] = 1.0                                    # the newest input alone
    y = la.causal_conv(x, w, activation="silu")
    _relative(x.double(), y.double(), _silu(x.double()), dtype, 9)
    state = torch.zeros(2048, 1, 64, device=DEV, dtype=dtype)
    y = la.causal_conv_step(state, x[0], w, activation="silu")
    _relative(x[0].double(), y.double(), _silu(x[0].double()), dtype, 9)
    # a scan whose state stays 0, so that its output is skip·x·silu(gate), with x = skip = 1
    one, zero = torch.ones_like(x), torch.zeros(1, 2048, 16, device=DEV, dtype=dtype)
    a, skip = -torch.ones(64, 16, device=DEV), torch.ones(64, device=DEV)
    y = la.selective_scan(one, one, a, zero, zero, skip=skip, gate=x)
    _relative(x.double(), y.double(), _silu(x.double()), dtype, 9 + 2)
    y = la.selective_step(torch.zeros(2048, 64, 16, device=DEV), one[0], one[0], a, zero[0], zero[0],
                          skip=skip, gate=x[0])
    _relative(x[0].double(), y.double(), _silu(x[0].double()), dtype, 9 + 2)


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
def test_relative_accuracy_of_the_step_size(dtype):
    """softplus(dt) read back from a state: h = Δ·x·b with x = b = 1 and no state before."""
    dt = torch.linspace(-80, 80, 64 * 2048, device=DEV).to(dtype).view(2048, 1, 64)
    one, b = torch.ones_like(dt), torch.ones(2048, 1, 16, device=DEV, dtype=dtype)
    a = -torch.ones(64, 16, device=DEV)
    want = _softplus(dt.double())[:, 0, :, None].expand(2048, 64, 16)
    x = dt.double()[:, 0, :, None].expand(2048, 64, 16)
    _, h = la.selective_scan(one, dt, a, b, b, return_state=True)
    _relative(x, h.double(), want, torch.float32, 12 + 2)
    h = torch.zeros(2048, 64, 16, device=DEV)
    la.selective_step(h, one[:, 0], dt[:, 0], a, b[:, 0], b[:, 0])
    _relative(x, h.double(), want, torch.float32, 12 + 2)


# ------------------------------------------------------------------ states that grow

@pytest.mark.parametrize("step,first,value", [
    (2.0, 2070, 1.0),          # e^160 over a chunk whose states are still 0
    (1.25, 1980, 1e-30)])      # e^100 over a chunk, from 1e-30 to 1e35
def test_scan_growth_over_chunks(step, first, value):
    """Positive rates: a chunk's factor can be past fp32's range while the states
    are not.  Every step's decay is off by at most (|Δ·a| + 3)·2^-24 relative (its
    argument, its 2^x), 120 steps of it: 4e-5."""
    n, D, S = 2100, 24, 16
    x = torch.zeros(1, n, D, device=DEV)
    x[:, first] = value
    dt = torch.full((1, n, D), step, device=DEV)
    a = torch.ones(D, S, device=DEV)
    a[:, 8:] = -1.0
    one = torch.ones(1, n, S, device=DEV)
    y, end = la.selective_scan(x, dt, a, one, one, softplus=False, return_state=True)
    h = torch.zeros(D, S, device=DEV, dtype=torch.float64)
    for t in range(n):
        h = torch.exp(step * a.double()) * h + step * x[0, t, :, None].double()
        if t in (first - 1, first, first + 20, n - 1):
            want = h.sum(-1)
            assert ((y[0, t].double() - want).abs() <= 4e-5 * want.abs()).all(), t
    assert ((end[0].double() - h).abs() <= 4e-5 * h.abs() + 1e-37).all()
    assert (y[:, :first] == 0).all()


# ------------------------------------------------------------------ outputs beside and over inputs

def test_outputs_beside_their_inputs_in_one_buffer():
    """Columns of one buffer that do not meet are let through, whatever lies between."""
    g = _gen(6)
    big = _randn(g, 3, 40, 384)
    keep = big.clone()
    w, cw = _randn(g, 64, 64, scale=0.125), _randn(g, 64, 4)
    x, out = big[..., 64:128], big[..., 128:192]
    want = la.causal_conv(x.clone(), cw)
    assert la.causal_conv(x, cw, out=out).data_ptr() == out.data_ptr() and torch.equal(out, want)
    want = la.linear(x.clone(), w)
    la.linear(x, w, out=out)
    assert torch.equal(out, want)
    i = dict(x=x, dt=big[..., :64], gate=big[..., 192:256], b=big[..., 256:272], c=big[..., 272:288],
             a=-torch.rand(64, 16, device=DEV, generator=g))
    want, end = la.selective_scan(**{k: v.clone() for k, v in i.items()}, return_state=True)
    got, after = la.selective_scan(**i, out=out, return_state=True)
    assert torch.equal(got, want) and torch.equal(after, end)
    one = {k: (v if k == "a" else v[:, 0]) for k, v in i.items()}
    s1, s2 = end.clone(), end.clone()
    want = la.selective_step(s1, **{k: v.clone() for k, v in one.items()})
    assert torch.equal(la.selective_step(s2, **one, out=big[:, 0, 320:]), want) and torch.equal(s1, s2)
    assert torch.equal(big[..., :128], keep[..., :128]) and torch.equal(big[:, 1:, 192:], keep[:, 1:, 192:])


@pytest.mark.parametrize("B,n,D", [(2, 33, 72), (4, 700, 2048), (1, 2100, 64)])
@pytest.mark.parametrize("over", ["x", "dt", "gate"])
def test_scan_output_may_be_an_input(B, n, D, over):
    g = _gen(7)
    i = dict(x=_randn(g, B, n, D), dt=_randn(g, B, n, D), gate=_randn(g, B, n, D), b=_randn(g, B, n, 16),
             c=_randn(g, B, n, 16), a=-torch.rand(D, 16, device=DEV, generator=g))
    want, end = la.selective_scan(**i, return_state=True)
    i[over] = i[over].clone()
    got, after = la.selective_scan(**i, out=i[over], return_state=True)
    assert torch.equal(got, want) and torch.equal(after, end)


def test_output_over_an_input_is_refused():
    g = _gen(8)
    x, w, cw = _randn(g, 2, 70, 64), _randn(g, 64, 64), _randn(g, 64, 4)
    i = dict(x=x, dt=_randn(g, 2, 70, 64), b=_randn(g, 2, 70, 16), c=_randn(g, 2, 70, 16),
             a=-torch.rand(64, 16, device=DEV, generator=g))
    wide = _randn(g, 2, 70, 192)
    before = la.launch_count()
    for f in (lambda: la.linear(x, w, out=x), lambda: la.causal_conv(x, cw, out=x),
              lambda: la.linear(x.view(-1, 64)[:64], w, out=w),
              lambda: la.causal_conv(wide[..., :64], cw, out=wide[..., 56:120]),
              lambda: la.selective_scan(**dict(i, x=wide[..., :64]), out=wide[..., 32:96]),
              lambda: la.selective_scan(**dict(i, b=wide[..., :16]), out=wide[..., 8:72])):
        with pytest.raises(la.LinAttnError):
            f()
    assert la.launch_count() == before


# ------------------------------------------------------------------ gradients

def _block_inputs(g, B=2, n=20, D=64):
    i = dict(x=_randn(g, B, n, D), dt=_randn(g, B, n, D), b=_randn(g, B, n, 16), c=_randn(g, B, n, 16),
             a=-torch.rand(D, 16, device=DEV, generator=g))
    return i, _randn(g, D, D, scale=0.125), _randn(g, D, 4)


def test_a_gradient_that_reaches_an_output_raises():
    i, w, cw = _block_inputs(_gen(9))
    one = {k: (v if k == "a" else v[:, 0].contiguous()) for k, v in i.items()}
    conv_state = torch.zeros(2, 3, 64, device=DEV, dtype=BF)
    state = torch.zeros(2, 64, 16, device=DEV)
    calls = {
        "linear": lambda p: la.linear(i["x"], p(w)),
        "causal_conv": lambda p: la.causal_conv(i["x"], p(cw), return_state=True),
        "causal_conv_step": lambda p: la.causal_conv_step(conv_state.clone(), one["x"], p(cw)),
        "selective_scan": lambda p: la.selective_scan(**dict(i, a=p(i["a"])), return_state=True),
        "selective_step": lambda p: la.selective_step(state.clone(), **dict(one, a=p(one["a"])))}
    for name, f in calls.items():
        plain = f(lambda t: t)
        leaf = []
        got = f(lambda t: leaf.append(t.clone().requires_grad_()) or leaf[0])
        with torch.no_grad():
            quiet = f(lambda t: leaf[0])
        plain, got, quiet = (v if isinstance(v, tuple) else (v,) for v in (plain, got, quiet))
        for p, q, r in zip(plain, got, quiet):
            assert torch.equal(p, q) and torch.equal(p, r)
            assert q.requires_grad and not r.requires_grad and not p.requires_grad
            with pytest.raises(RuntimeError, match=f"{name} has no backward"):
                (q.float() * 2).sum().backward(retain_graph=True)
        assert leaf[0].grad is None


def test_prompts_and_tokens_with_weights_that_require_gradients():
    """Without torch.no_grad(): the states that a prompt left are stepped as they are."""
    i, w, cw = _block_inputs(_gen(12))
    pw, pcw, pa = (t.clone().requires_grad_() for t in (w, cw, i["a"]))
    x, conv_state = la.causal_conv(la.linear(i["x"], pw), pcw, return_state=True)
    y, state = la.selective_scan(**dict(i, x=x, a=pa), return_state=True)
    for t in range(2):
        u = la.causal_conv_step(conv_state, la.linear(i["x"][:, t], pw), pcw)
        o = la.selective_step(state, u, i["dt"][:, t], pa, i["b"][:, t], i["c"][:, t])
    with torch.no_grad():
        x, conv_ref = la.causal_conv(la.linear(i["x"], w), cw, return_state=True)
        _, ref = la.selective_scan(**dict(i, x=x), return_state=True)
        for t in range(2):
            u = la.causal_conv_step(conv_ref, la.linear(i["x"][:, t], w), cw)
            want = la.selective_step(ref, u, i["dt"][:, t], i["a"], i["b"][:, t], i["c"][:, t])
    assert torch.equal(o, want) and torch.equal(state, ref) and torch.equal(conv_state, conv_ref)
    for v in (o, state, conv_state):
        with pytest.raises(RuntimeError, match="has no backward"):
            v.float().sum().backward(retain_graph=True)


def test_given_outputs_and_states_take_no_part_in_a_graph():
    i, w, cw = _block_inputs(_gen(10))
    p = w.clone().requires_grad_()
    out = torch.empty_like(i["x"])
    with pytest.raises(ValueError, match="no_grad"):
        la.linear(i["x"], p, out=out)
    with torch.no_grad():
        assert torch.equal(la.linear(i["x"], p, out=out), la.linear(i["x"], w))
    one = {k: (v if k == "a" else v[:, 0].contiguous()) for k, v in i.items()}
    state = torch.zeros(2, 64, 16, device=DEV, requires_grad=True)
    with pytest.raises(ValueError, match="state"):
        la.selective_step(state, **one)
    with pytest.raises(ValueError, match="state"):
        la.causal_conv_step(torch.zeros(2, 3, 64, device=DEV, dtype=BF, requires_grad=True), one["x"], cw)
    # one that comes from another operator would keep a graph that no longer holds
    with pytest.raises(ValueError, match="state"):
        la.selective_step(state * 2, **one)
    # written in place: a graph that has kept the old values notices
    for s, write in ((torch.zeros(2, 64, 16, device=DEV), lambda s: la.selective_step(s, **one)),
                     (torch.zeros_like(i["x"]), lambda s: la.selective_scan(**i, out=s))):
        q = torch.ones_like(s, requires_grad=True)
        loss = (q * s).sum()
        write(s)
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    with torch.inference_mode():         # nothing keeps versions there
        s = torch.zeros(2, 64, 16, device=DEV)
        la.selective_step(s, **one)
        la.linear(i["x"], p, out=torch.empty_like(i["x"]))


# ------------------------------------------------------------------ every kernel, at sizes that it is chosen for

@pytest.mark.parametrize("kernel,m,k,n", [
    ("few16", 11, 208, 264), ("few16", 16, 4096, 160), ("few32", 537, 384, 96), ("few32", 37, 208, 344),
    ("few64", 604, 328, 1088), ("few64", 175, 1744, 2520), ("few128", 1499, 192, 1208),
    ("few128", 1170, 1224, 1400), ("pair128", 2619, 352, 1608), ("pair128", 6421, 64, 528),
    ("pair128", 12611, 112, 376), ("pair256", 9803, 64, 144), ("pair256", 8905, 144, 376),
    ("rows2", 2, 604, 4100), ("rows8", 41, 476, 1588), ("tile8x1", 4095, 164, 1164),
    ("tile8x2", 1290, 156, 916), ("tile8x2", 2315, 616, 816), ("tile8x4", 723, 236, 1076),
    ("tile4x1", 3287, 76, 268), ("tile4x1", 275, 1428, 4092), ("tile4x2", 214, 828, 1692),
    ("tile4x4", 97, 2044, 1404)])
@pytest.mark.parametrize("act,use_bias,use_res", [("none", False, False), ("silu", True, True)])
def test_linear_kernel(kernel, m, k, n, act, use_bias, use_res):
    dtype = torch.float32 if kernel[:4] in ("rows", "tile") else BF
    assert la.selftest_linear_kernel(dtype, m, n, k) == kernel
    g = _gen(m + n)
    big = _randn(g, m, n + 16, dtype=dtype)           # the output's columns of a wider buffer
    keep = big.clone()
    x, w = _randn(g, m, k, dtype=dtype), _randn(g, n, k, dtype=dtype, scale=k ** -0.5)
    bias = _randn(g, n, dtype=dtype) if use_bias else None
    res = _randn(g, m, n, dtype=dtype) if use_res else None
    out = big[:, 8:8 + n]
    y = la.linear(x, w, bias=bias, activation=act, residual=res, out=out)
    ref, ab = _linear_ref(x, w, bias, act, res)
    _close(y, ref, ab, k + 2, dtype, kernel)
    assert torch.equal(big[:, :8], keep[:, :8]) and torch.equal(big[:, 8 + n:], keep[:, 8 + n:])
    assert torch.equal(y, la.linear(x, w, bias=bias, activation=act, residual=res))
    assert la.last_device_status() == 0


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("B", [301, 302, 303])
def test_step_four_entries_per_lane_and_a_remainder(dtype, S, B):
    D = 2040
    assert la.selftest_step_kernel(B, D, S) == "step4"
    i = _scan_inputs(_gen(S + B), B, 1, D, S, dtype, state=True)
    y, ys, h, hs = _scan_ref(i)
    one = {k: (v[:, 0] if k in ("x", "dt", "b", "c", "gate") else v) for k, v in i.items()}
    room = torch.full((B + 1, D, S), 7.0, device=DEV)          # nothing past the last entry is written
    st = room[:B].copy_(one.pop("state"))
    got = la.selective_step(st, **one)
    _close(got, y[:, 0], 4 * ys[:, 0], S + 1, dtype, "y")
    _close(st, h, 4 * hs, S + 1, torch.float32, "state")
    assert (room[B] == 7.0).all()
