"""Gated-delta block operators, host side: refusals before anything is queued
(no GPU needed)."""
import ctypes

import pytest
import torch

import causal_kernelized_linear_gb300 as la
from causal_kernelized_linear_gb300 import _binding as B

OK, BAD, UNS = B.LA_OK, B.LA_ERR_INVALID_ARG, B.LA_ERR_UNSUPPORTED
BF16, F32, E4M3 = B.LA_BF16, B.LA_F32, B.LA_E4M3
BASE = 0x7f0000000000   # of made-up device addresses, far apart


@pytest.fixture(scope="module", autouse=True)
def lib():
    la.build()
    return la.load()


def at(i):
    return BASE + i * (1 << 36)


def heads(i, b=2, n=8, h=2, d=64, dtype=BF16, sb=None, sn=None, sh=None, ptr=None):
    sh = d if sh is None else sh
    sn = h * sh if sn is None else sn
    return B.LaHeads(at(i) if ptr is None else ptr, dtype, b, n, h, d, n * sn if sb is None else sb, sn, sh)


def rows(i, b=1, n=8, d=64, dtype=BF16, sb=None, sn=None, ptr=None):
    sn = d if sn is None else sn
    return B.LaRows(at(i) if ptr is None else ptr, dtype, b, n, d, n * sn if sb is None else sb, sn)


def ref(r):
    return ctypes.byref(r) if r is not None else None


def delta(n=8, b=2, **kw):
    """la_gated_delta on a call that is right but for `kw`."""
    g = {"q": heads(0, b, n), "k": heads(1, b, n), "v": heads(2, b, n, 4), "dt": rows(3, b, n, 4), "a": at(4),
         "beta": rows(5, b, n, 4), "bias": at(6), "scale": 1.0, "sin": at(7), "lens": at(8), "out": heads(9, b, n, 4),
         "sout": at(10), **kw}
    return la.load().la_gated_delta(ref(g["q"]), ref(g["k"]), ref(g["v"]), ref(g["dt"]), g["a"], ref(g["beta"]),
                                    g["bias"], 1, 1, 1, g["scale"], g["sin"], g["lens"], ref(g["out"]), g["sout"], None)


def test_gated_delta_refusals():
    assert delta(b=0) == OK                                          # nothing to do, and all the rest is right
    for name in ("q", "k", "v", "dt", "a", "beta", "out"):
        assert delta(**{name: None}) == BAD, name
    assert delta(k=heads(1, d=72)) == BAD                            # dk differs
    assert delta(k=heads(1, h=4)) == BAD and delta(k=heads(1, n=9)) == BAD
    assert delta(v=heads(2, h=3), out=heads(9, h=3), dt=rows(3, 2, 8, 3), beta=rows(5, 2, 8, 3)) == BAD   # 3 % 2
    assert delta(out=heads(9, h=2)) == BAD and delta(out=heads(9, h=4, d=72)) == BAD
    assert delta(out=heads(9, h=4, dtype=F32)) == BAD and delta(q=heads(0, dtype=F32)) == BAD
    assert delta(q=heads(0, dtype=E4M3)) == BAD and delta(q=heads(0, dtype=9)) == BAD
    assert delta(dt=rows(3, 2, 8, 3)) == BAD and delta(beta=rows(5, 2, 7, 4)) == BAD
    assert delta(dt=rows(3, 2, 8, 4, F32)) == BAD                    # beta of another type
    assert delta(dt=rows(3, 2, 8, 4, E4M3), beta=rows(5, 2, 8, 4, E4M3)) == BAD
    f = {"q": heads(0, dtype=F32), "k": heads(1, dtype=F32), "v": heads(2, h=4, dtype=F32), "out": heads(9, h=4, dtype=F32)}
    assert delta(**f) == BAD                                         # fp32 with gates in bf16
    assert delta(b=0, dt=rows(3, 0, 8, 4, F32, ptr=4), beta=rows(5, 0, 8, 4, F32)) == OK
    assert delta(q=heads(0, ptr=at(0) + 8)) == BAD and delta(q=heads(0, ptr=0)) == BAD
    assert delta(q=heads(0, sh=68)) == BAD and delta(k=heads(1, sn=132)) == BAD and delta(v=heads(2, h=4, sb=2052)) == BAD
    assert delta(q=heads(0, sn=-128)) == BAD
    assert delta(dt=rows(3, 2, 8, 4, ptr=at(3) + 1)) == BAD          # off an element
    assert delta(a=at(4) + 4) == BAD and delta(bias=at(6) + 8) == BAD and delta(lens=at(8) + 2) == BAD
    assert delta(sin=at(7) + 4) == BAD and delta(sout=at(10) + 4) == BAD
    assert delta(scale=float("nan")) == BAD and delta(scale=float("inf")) == BAD
    # outputs that lie on themselves
    assert delta(out=heads(9, h=4, sh=0)) == BAD and delta(out=heads(9, h=4, sn=64)) == BAD
    assert delta(out=heads(9, h=4, sb=512)) == BAD
    # sizes
    for d, st in ((4, BAD), (12, BAD), (264, UNS)):
        assert delta(q=heads(0, d=d), k=heads(1, d=d)) == st, d
    assert delta(v=heads(2, h=4, d=520), out=heads(9, h=4, d=520)) == UNS
    assert delta(**{**f, "q": heads(0, dtype=F32, d=12), "k": heads(1, dtype=F32, d=12)},
                 dt=rows(3, 2, 8, 4, F32), beta=rows(5, 2, 8, 4, F32)) == UNS


def test_gated_delta_refuses_shared_memory():
    assert delta(sout=at(7)) == BAD and delta(sout=at(7) + 4096) == BAD          # the state before
    assert delta(out=heads(2, h=4)) == BAD and delta(out=heads(0, h=4)) == BAD   # v, q
    assert delta(sout=at(2)) == BAD and delta(sout=at(0) + 512) == BAD and delta(sout=at(3)) == BAD
    assert delta(sout=at(4)) == BAD and delta(sout=at(6)) == BAD and delta(sout=at(8)) == BAD
    assert delta(sin=at(9)) == BAD and delta(sout=at(9)) == BAD and delta(lens=at(9)) == BAD
    assert delta(a=at(9)) == BAD and delta(bias=at(9) + 64) == BAD
    # parts of one buffer that lie between one another are apart; the same part is not
    sn = 1024
    v = heads(2, h=4, sn=sn)
    beside, on = heads(2, h=4, sn=sn, ptr=at(2) + 2 * 256), heads(2, h=4, sn=sn, ptr=at(2) + 2 * 64)
    assert delta(v=v, out=on) == BAD
    assert delta(b=0, v=heads(2, 0, h=4, sn=sn), out=heads(2, 0, h=4, sn=sn)) == OK
    swap = {"sh": 8 * 64, "sn": 64, "sb": 4 * 8 * 64}                # [B, H, n, d]
    assert delta(v=heads(2, h=4, **swap), out=heads(2, h=4, **swap)) == BAD
    apart = heads(2, h=4, sb=2 * 8 * sn, sn=2 * sn, sh=128, ptr=at(2) + 2 * 64)
    assert beside.data != on.data and apart.data == on.data


def step(**kw):
    g = {"state": at(7), "q": heads(0, 2, 1), "k": heads(1, 2, 1), "v": heads(2, 2, 1, 4), "dt": rows(3, 2, 1, 4),
         "a": at(4), "beta": rows(5, 2, 1, 4), "bias": None, "out": heads(9, 2, 1, 4), **kw}
    return la.load().la_gated_delta_step(g["state"], ref(g["q"]), ref(g["k"]), ref(g["v"]), ref(g["dt"]), g["a"],
                                         ref(g["beta"]), g["bias"], 1, 1, 1, 1.0, ref(g["out"]), None)


def test_gated_delta_step_refusals():
    none = {"q": heads(0, 0, 1), "k": heads(1, 0, 1), "v": heads(2, 0, 1, 4), "dt": rows(3, 0, 1, 4),
            "beta": rows(5, 0, 1, 4), "out": heads(9, 0, 1, 4)}
    assert step(**none) == OK and step(state=None, **none) == OK
    assert step(state=None) == BAD and step(state=at(7) + 8) == BAD
    two = {"q": heads(0, 2, 2), "k": heads(1, 2, 2), "v": heads(2, 2, 2, 4), "dt": rows(3, 2, 2, 4),
           "beta": rows(5, 2, 2, 4), "out": heads(9, 2, 2, 4)}
    assert step(**two) == BAD                                        # two tokens
    assert step(state=at(0)) == BAD and step(state=at(2)) == BAD and step(state=at(9)) == BAD
    assert step(state=at(3)) == BAD and step(state=at(4)) == BAD
    assert step(out=heads(2, 2, 1, 4)) == BAD


def norm(group=64, eps=1e-6, **kw):
    g = {"x": rows(0), "w": at(1), "res": None, "gate": None, "out": rows(2), "scale": None, "sum": None, **kw}
    return la.load().la_rms_norm(ref(g["x"]), g["w"], group, eps, ref(g["res"]), ref(g["gate"]), ref(g["out"]),
                                 g["scale"], ref(g["sum"]), None)


def test_rms_norm_refusals():
    empty = {"x": rows(0, n=0), "out": rows(2, n=0)}
    assert norm(**empty) == OK
    assert norm(x=rows(0, n=0), out=rows(2, n=0, dtype=E4M3)) == OK
    assert norm(x=None) == BAD and norm(out=None) == BAD
    assert norm(out=rows(2, n=9)) == BAD and norm(out=rows(2, d=72)) == BAD and norm(out=rows(2, dtype=F32)) == BAD
    assert norm(x=rows(0, dtype=E4M3), out=rows(2, dtype=E4M3), scale=at(3)) == BAD
    assert norm(x=rows(0, b=2), out=rows(2, b=2)) == BAD
    assert norm(group=0) == BAD and norm(group=-64) == BAD and norm(group=48) == BAD and norm(group=4) == BAD
    assert norm(group=128) == BAD
    assert norm(eps=-1e-6) == BAD and norm(eps=float("nan")) == BAD and norm(eps=float("inf")) == BAD
    assert norm(w=at(1) + 8) == BAD
    assert norm(out=rows(2, dtype=E4M3)) == BAD                      # 8 bits without scales
    assert norm(scale=at(3)) == BAD                                  # scales without 8 bits
    assert norm(out=rows(2, dtype=E4M3), scale=at(3) + 2) == BAD
    assert norm(out=rows(2, dtype=E4M3, sn=68), scale=at(3)) == BAD  # off 8 bytes
    assert norm(sum=rows(4)) == BAD                                  # a sum of nothing
    f = {"x": rows(0, d=60, dtype=F32), "out": rows(2, d=60, dtype=E4M3), "scale": at(3)}
    assert norm(group=60, **f) == BAD                                # 8 bits want multiples of 8
    assert norm(res=rows(4, n=7)) == BAD and norm(gate=rows(4, d=72)) == BAD and norm(gate=rows(4, dtype=F32)) == BAD
    assert norm(out=rows(2, sn=32)) == BAD and norm(out=rows(2, sn=0)) == BAD
    wide = 65536 + 8
    assert norm(group=wide, x=rows(0, d=wide), out=rows(2, d=wide)) == UNS
    many = (1 << 30) + 1
    assert norm(x=rows(0, n=many), out=rows(2, n=many)) == UNS


def test_rms_norm_refuses_shared_memory():
    assert norm(out=rows(1)) == BAD                                  # the weight
    assert norm(out=rows(0, ptr=at(0) + 16, sn=64)) == BAD           # x, but for 8 features
    assert norm(gate=rows(5), out=rows(5, ptr=at(5) + 128)) == BAD
    assert norm(out=rows(0, dtype=E4M3), scale=at(3)) == BAD         # 8 bits over 16
    assert norm(out=rows(2, dtype=E4M3), scale=at(2) + 64) == BAD and norm(out=rows(2, dtype=E4M3), scale=at(0)) == BAD
    assert norm(out=rows(2, dtype=E4M3), scale=at(1)) == BAD
    r = {"res": rows(4)}
    assert norm(sum=rows(2), **r) == BAD                             # sum and out
    assert norm(sum=rows(5), gate=rows(5), **r) == BAD
    assert norm(sum=rows(1), **r) == BAD
    assert norm(sum=rows(0, ptr=at(0) + 16), **r) == BAD


def lin8(**kw):
    g = {"x": rows(0, n=8, d=64, dtype=E4M3), "xs": at(1), "w": rows(2, n=32, d=64, dtype=E4M3), "ws": at(3),
         "bias": None, "act": 0, "res": None, "out": rows(4, n=8, d=32), **kw}
    return la.load().la_linear_e4m3(ref(g["x"]), g["xs"], ref(g["w"]), g["ws"], g["bias"], g["act"], ref(g["res"]),
                                    ref(g["out"]), None)


def test_linear_e4m3_refusals():
    assert lin8(x=rows(0, n=0, d=64, dtype=E4M3), xs=None, out=rows(4, n=0, d=32)) == OK
    for name in ("x", "xs", "w", "ws", "out"):
        assert lin8(**{name: None}) == BAD, name
    assert lin8(x=rows(0)) == BAD and lin8(w=rows(2, n=32)) == BAD   # bf16 operands
    assert lin8(out=rows(4, d=32, dtype=F32)) == BAD and lin8(out=rows(4, d=32, dtype=E4M3)) == BAD
    assert lin8(res=rows(5, d=32, dtype=F32)) == BAD
    assert lin8(x=rows(0, d=80, dtype=E4M3)) == BAD                  # K differs
    assert lin8(out=rows(4, n=9, d=32)) == BAD and lin8(out=rows(4, d=40)) == BAD
    k = {"x": rows(0, d=72, dtype=E4M3), "w": rows(2, n=32, d=72, dtype=E4M3)}
    assert lin8(**k) == BAD                                          # K off 16
    assert lin8(w=rows(2, n=36, d=64, dtype=E4M3), out=rows(4, d=36)) == BAD
    assert lin8(x=rows(0, dtype=E4M3, ptr=at(0) + 8)) == BAD and lin8(x=rows(0, dtype=E4M3, sn=72)) == BAD
    assert lin8(x=rows(0, dtype=E4M3, sn=0)) == BAD                  # rows overlap
    assert lin8(xs=at(1) + 2) == BAD and lin8(ws=at(3) + 4) == BAD and lin8(bias=at(6) + 8) == BAD
    assert lin8(act=5) == BAD and lin8(res=rows(5, n=7, d=32)) == BAD
    for name, p in (("xs", at(4)), ("ws", at(4)), ("bias", at(4) + 16)):
        assert lin8(**{name: p}) == BAD                              # the output over a parameter
    assert lin8(out=rows(0, n=8, d=32)) == BAD and lin8(res=rows(4, n=8, d=32, ptr=at(4) + 16)) == BAD
    many = (1 << 30) + 1
    assert lin8(x=rows(0, n=many, dtype=E4M3), out=rows(4, n=many, d=32)) == UNS


def test_python_refusals():
    x = torch.zeros(2, 3, 2, 64)
    g = torch.zeros(2, 3, 2)
    a = torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        la.gated_delta(x, x, x, g, a, g)
    with pytest.raises(ValueError, match="4 axes"):
        la.gated_delta(x[0], x, x, g, a, g)
    with pytest.raises(ValueError, match="3 axes"):
        la.gated_delta_step(torch.zeros(2, 2, 64, 64), x, x, x, g, a, g)
    with pytest.raises(ValueError, match="unsupported dtype"):
        la.gated_delta(x.half(), x, x, g, a, g)
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        la.gated_delta(None, x, x, g, a, g)
    with pytest.raises(ValueError, match="CUDA tensor"):
        la.rms_norm(x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        la.linear_e4m3(x[0, 0].to(torch.float8_e4m3fn), a, x[0, 0].to(torch.float8_e4m3fn), a)
    with pytest.raises(TypeError, match="x must be"):
        la.rms_norm("x")
