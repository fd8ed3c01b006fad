"""What a NaN or infinity of a token reaches in the gated delta rule: its own outputs and
what comes after it, and of a value no other column.  In bf16 the tokens go in chunks of
64, of which the earlier ones must not see it."""
import pytest
import torch

import causal_kernelized_linear_gb300 as la
from test_delta_block_gpu import BF16, CHUNKED, DEV, DTYPES, F32, IDS, _call, _check, _gen, _inputs, _randn

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
SIZES = [(150, 64, 64, 70), (150, 64, 64, 127), (130, 128, 136, 64), (64, 128, 128, 63), (40, 40, 72, 1), (100, 128, 256, 0)]
SIZE_IDS = ["x".join(map(str, s)) for s in SIZES]


def _to(x, n):
    return {k: (v[:, :n] if v.dim() > 1 else v) for k, v in x.items()}


def _before(got, x, t, **kw):
    """The outputs of the tokens before t against 64 bits."""
    if t:
        part = _to(x, t)
        _, after = _call(part, **kw)   # (checked with them; a call of its own)
        _check((got[0][:, :t], after), part, **kw)


def _bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF16 else torch.int32)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("n,dk,dv,t", SIZES, ids=SIZE_IDS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_a_value_reaches_its_column(dtype, n, dk, dv, t, value):
    x = _inputs(2, n, 1, 2, dk, dv, dtype, seed=n + t)
    state = _randn(_gen(t), 2, 2, dk, dv, scale=0.3)
    clean = {k: v.clone() for k, v in x.items()}
    ref = _call(clean, state=state)
    col = dv - 3
    x["v"][0, t, 1, col] = value
    got = _call(x, state=state)
    _before(got, clean, t, state=state)
    # the other columns go on as if nothing had been; `whole` has the clean ones in its place
    whole = [g.clone() for g in got]
    whole[0][0, t:, 1, col], whole[1][0, 1, :, col] = ref[0][0, t:, 1, col], ref[1][0, 1, :, col]
    assert torch.isfinite(whole[0]).all() and torch.isfinite(whole[1]).all()
    _check(whole, clean, state=state)
    assert not torch.isfinite(got[0][0, t:, 1, col]).any() and not torch.isfinite(got[1][0, 1, :, col]).any()
    # other heads and sequences are the same bits
    assert torch.equal(got[0][1], ref[0][1]) and torch.equal(got[0][0, :, 0], ref[0][0, :, 0])
    assert torch.equal(got[1][1], ref[1][1]) and torch.equal(got[1][0, 0], ref[1][0, 0])
    again = _call(x, state=state)
    assert torch.equal(_bits(again[0]), _bits(got[0])) and torch.equal(_bits(again[1]), _bits(got[1]))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("n,dk,dv,t", SIZES, ids=SIZE_IDS)
@pytest.mark.parametrize("name,value", [("k", NAN), ("k", INF), ("dt", NAN), ("beta", NAN)])
def test_a_key_or_gate_reaches_what_follows(dtype, n, dk, dv, t, name, value):
    x = _inputs(1, n, 2, 2, dk, dv, dtype, seed=n + t)
    clean = {k: v.clone() for k, v in x.items()}
    ref = _call(clean)
    at = (0, t, 1, dk - 1) if name == "k" else (0, t, 1)
    x[name][at] = value
    got = _call(x)
    _before(got, clean, t)
    assert torch.equal(got[0][:, :, 0], ref[0][:, :, 0]) and torch.equal(got[1][:, 0], ref[1][:, 0])
    assert torch.isnan(got[0][0, t:, 1]).all() and torch.isnan(got[1][0, 1]).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("n,dk,dv,t", SIZES, ids=SIZE_IDS)
def test_a_query_reaches_its_output_alone(dtype, n, dk, dv, t):
    x = _inputs(1, n, 1, 2, dk, dv, dtype, seed=n + t)
    ref = _call(x)
    x["q"][0, t, 0, 5] = NAN
    got = _call(x)
    assert torch.isnan(got[0][0, t]).all() and torch.equal(got[1], ref[1])
    rest = [i for i in range(n) if i != t]
    assert torch.equal(got[0][:, rest], ref[0][:, rest])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_infinite_gates_have_values(dtype):
    # a step of +inf clears the state, one of −inf leaves it; a strength of ±inf is 1 or 0
    x = _inputs(1, 140, 1, 1, 64, 64, dtype, seed=3)
    state = _randn(_gen(1), 1, 1, 64, 64)
    x["dt"][0, [5, 70, 100]] = INF
    x["dt"][0, [6, 80]] = -INF
    x["beta"][0, [7, 90]] = INF
    x["beta"][0, [8, 91]] = -INF
    _check(_call(x, state=state), x, state=state)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("dk", [64, 128])
def test_several_spoilt_values(dtype, dk):
    # in one chunk and in later ones, some of a column that is spoilt already
    x = _inputs(1, 300, 1, 1, dk, 136, dtype, seed=5)
    clean = {k: v.clone() for k, v in x.items()}
    ref = _call(clean)
    spoilt = {3: 70, 131: 90, 60: 129, 61: 192, 4: 299}   # column: first token
    for col, t in spoilt.items():
        x["v"][0, t, 0, col] = NAN
    x["v"][0, 200, 0, 3] = INF
    out, state = _call(x)
    for col, t in spoilt.items():
        assert torch.isnan(out[0, t:, 0, col]).all() and torch.isnan(state[0, 0, :, col]).all()
        out[0, t:, 0, col], state[0, 0, :, col] = ref[0][0, t:, 0, col], ref[1][0, 0, :, col]
    _check((out, state), clean)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_padding_that_holds_nan_without_lengths(dtype):
    lens = [200, 1, 64, 65, 130, 199]
    x = _inputs(len(lens), 200, 1, 2, 64, 128, dtype, seed=7)
    clean = {k: v.clone() for k, v in x.items()}
    ref = _call(clean)
    for i, l in enumerate(lens):
        for name in ("q", "k", "v", "dt", "beta"):
            x[name][i, l:] = NAN
    out, state = _call(x)
    for i, l in enumerate(lens):
        assert torch.isnan(out[i, l:]).all()
        out[i, l:], state[i] = ref[0][i, l:], ref[1][i]
    _check((out, state), clean)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("partial", [False, True])
def test_ragged_sequences_with_a_spoilt_value(dtype, partial):
    # outputs behind a sequence are zero, within its last chunk too, and what is beside it is kept
    n, live = 150, 100 if partial else 128
    x = _inputs(1, n, 1, 2, 128, 72, dtype, seed=8)
    clean = {k: v.clone() for k, v in x.items()}
    lengths = torch.tensor([live], device=DEV, dtype=torch.int32)
    ref = _call(clean, lengths=lengths)
    x["v"][0, 80, 1, 7] = NAN
    x["k"][0, live:], x["v"][0, live:] = NAN, INF
    big = torch.full((1, n + 2, 2, 88), 7.0, device=DEV, dtype=dtype)
    out, state = _call(x, lengths=lengths, out=big[:, 1:-1, :, 8:80])
    assert (out[0, live:] == 0).all() and torch.isnan(out[0, 80:live, 1, 7]).all()
    out[0, 80:live, 1, 7], state[0, 1, :, 7] = ref[0][0, 80:live, 1, 7], ref[1][0, 1, :, 7]
    _check((out, state), clean, lengths=lengths)
    for edge in (big[:, 0], big[:, -1], big[..., :8], big[..., 80:]):
        assert (edge == 7).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_a_spoilt_state(dtype):
    # a column of the state that enters; and a state that overflows on the way
    x = _inputs(1, 200, 1, 1, 64, 64, dtype, seed=9)
    state = _randn(_gen(1), 1, 1, 64, 64)
    ref = _call(x, state=state)
    bad = state.clone()
    bad[0, 0, 10, 20] = INF
    out, after = _call(x, state=bad)
    assert not torch.isfinite(out[..., 20]).any() and not torch.isfinite(after[0, 0, :, 20]).any()
    out[..., 20], after[..., 20] = ref[0][..., 20], ref[1][..., 20]
    _check((out, after), x, state=state)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_parts_with_spoilt_values(dtype):
    x = _inputs(1, 2500, 1, 1, 64, 64, dtype, seed=3)
    x["a"] = x["a"] * 0.002
    clean = {k: v.clone() for k, v in x.items()}
    ref = _call(clean)
    spoilt = {3: 1500, 9: 1510, 40: 2400}
    for col, t in spoilt.items():
        x["v"][0, t, 0, col] = NAN
    out, state = _call(x)
    for col, t in spoilt.items():
        assert torch.isnan(out[0, t:, 0, col]).all() and torch.isnan(state[0, 0, :, col]).all()
        out[0, t:, 0, col], state[0, 0, :, col] = ref[0][0, t:, 0, col], ref[1][0, 0, :, col]
    _check((out, state), clean, parts=True)
    x = {k: v.clone() for k, v in clean.items()}
    x["k"][0, 1300, 0, 1] = NAN
    out, state = _call(x)
    assert torch.isfinite(out[0, :1300]).all() and torch.isnan(out[0, 1300:]).all() and torch.isnan(state).all()
    out[0, 1300:] = ref[0][0, 1300:]
    _check((out, ref[1]), clean, parts=True)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_growth_past_the_range_of_fp32(dtype):
    # steps below zero: e^192 over a chunk whose state is zero, and e^30 once it is not
    x = _inputs(1, 150, 1, 2, 64, 64, dtype, seed=6, gates=F32)
    x["dt"] = torch.full_like(x["dt"], -1.0)
    x["a"] = torch.tensor([-3.0, -2.5], device=DEV)
    x["dt_bias"] = None
    x["beta"] = torch.rand(x["beta"].shape, device=DEV, generator=_gen(1))
    x["beta"][:, :140] = 0
    kw = {"softplus": False, "sigmoid": False}
    _check(_call(x, **kw), x, how=CHUNKED, **kw)
    assert la.last_device_status() == 0
