"""State-space block operators, host side: refusals before anything is queued
(no GPU needed)."""
import ctypes

import pytest
import torch

import causal_kernelized_linear_gb300 as la
from causal_kernelized_linear_gb300 import _binding as B

OK, BAD, UNS = B.LA_OK, B.LA_ERR_INVALID_ARG, B.LA_ERR_UNSUPPORTED
P0 = 0x10000


@pytest.fixture(scope="module", autouse=True)
def lib():
    la.build()
    return la.load()


def rows(b=1, n=8, d=64, ptr=P0, dtype=B.LA_BF16, sb=None, sn=None):
    sn = d if sn is None else sn
    return B.LaRows(ptr, dtype, b, n, d, n * sn if sb is None else sb, sn)


def ref(r):
    return ctypes.byref(r) if r is not None else None


def lin(x=None, w=None, bias=None, act=0, res=None, out=None):
    x, w = x or rows(n=8, d=64), w or rows(n=32, d=64)
    return la.load().la_linear(ref(x), ref(w), bias, act, ref(res),
                              ref(out or rows(n=8, d=32)), None)


def test_linear_refusals():
    assert la.load().la_linear(None, ref(rows()), None, 0, None, ref(rows()), None) == BAD
    assert la.load().la_linear(ref(rows()), None, None, 0, None, ref(rows()), None) == BAD
    assert la.load().la_linear(ref(rows()), ref(rows()), None, 0, None, None, None) == BAD
    assert lin(x=rows(d=72)) == BAD                            # K differs
    assert lin(out=rows(n=9, d=32)) == BAD                     # M differs
    assert lin(out=rows(n=8, d=40)) == BAD                     # N differs
    assert lin(out=rows(n=8, d=32, dtype=B.LA_F32)) == BAD     # dtype differs
    assert lin(x=rows(dtype=7)) == BAD
    assert lin(x=rows(b=2)) == BAD                             # a batch
    assert lin(x=rows(ptr=P0 + 8)) == BAD                      # misaligned data
    assert lin(x=rows(ptr=0)) == BAD
    assert lin(x=rows(sn=68)) == BAD                           # row stride off 16 bytes
    assert lin(x=rows(sn=-64)) == BAD
    assert lin(x=rows(sn=0)) == BAD and lin(w=rows(n=32, sn=32)) == BAD   # rows overlap
    assert lin(out=rows(n=8, d=32, sn=16)) == BAD
    assert lin(bias=P0 + 4) == BAD
    assert lin(act=5) == BAD and lin(act=-1) == BAD
    assert lin(res=rows(n=7, d=32)) == BAD
    assert lin(x=rows(d=60), w=rows(n=32, d=60)) == BAD        # K off 16 bytes
    big = rows(n=(1 << 30) + 1)
    assert lin(x=big, out=rows(n=(1 << 30) + 1, d=32)) == UNS
    assert lin(x=rows(n=0), out=rows(n=0, d=32)) == OK         # nothing to do


def conv(x=None, w=0x20000, width=4, bias=None, act=2, sin=None, lens=None, out=None, sout=None):
    x = x or rows(b=2)
    return la.load().la_causal_conv(ref(x), w, width, bias, act, sin, lens,
                                   ref(out or rows(b=2)), sout, None)


def test_conv_refusals():
    assert la.load().la_causal_conv(None, P0, 4, None, 2, None, None, ref(rows()), None, None) == BAD
    assert conv(w=None) == BAD and conv(w=0x20004) == BAD
    assert conv(width=1) == UNS and conv(width=5) == UNS
    assert conv(act=1) == UNS and conv(act=9) == BAD
    assert conv(bias=0x30002) == BAD
    assert conv(out=rows(b=2, n=9)) == BAD and conv(out=rows(b=3)) == BAD
    assert conv(out=rows(b=2, dtype=B.LA_F32)) == BAD
    assert conv(out=rows(b=2, sb=64)) == BAD                   # batch entries coincide
    assert conv(out=rows(b=2, sn=0, sb=512)) == BAD
    assert conv(x=rows(b=2, sb=100)) == BAD
    assert conv(x=rows(b=2, d=68), out=rows(b=2, d=68)) == BAD
    assert conv(sin=0x30008) == BAD and conv(sout=0x30008) == BAD
    assert conv(lens=0x30002) == BAD
    assert conv(sin=0x30000, sout=0x30100) == BAD              # the states overlap
    assert conv(x=rows(b=2, d=(1 << 20) + 8), out=rows(b=2, d=(1 << 20) + 8)) == UNS
    assert conv(x=rows(b=0), out=rows(b=0)) == OK


def test_conv_step_refusals():
    f = la.load().la_causal_conv_step
    one = rows(b=2, n=1)
    assert f(None, ref(one), 0x20000, 4, None, 2, ref(one), None) == BAD
    assert f(0x30004, ref(one), 0x20000, 4, None, 2, ref(one), None) == BAD
    assert f(0x30000, ref(rows(b=2, n=2)), 0x20000, 4, None, 2, ref(rows(b=2, n=2)), None) == BAD
    assert f(0x30000, ref(one), 0x20000, 6, None, 2, ref(one), None) == UNS


def scan(x=None, dt=None, a=0x20000, S=16, b=None, c=None, skip=None, gate=None, bias=None,
         sin=None, lens=None, out=None, sout=None):
    return la.load().la_selective_scan(
        ref(x or rows(b=2)), ref(dt or rows(b=2)), a, S, ref(b or rows(b=2, d=16)),
        ref(c or rows(b=2, d=16)), skip, ref(gate), bias, 1, sin, lens, ref(out or rows(b=2)),
        sout, None)


def test_scan_refusals():
    assert scan(a=None) == BAD and scan(a=0x20008) == BAD
    assert scan(dt=rows(b=2, n=9)) == BAD and scan(gate=rows(b=2, n=9)) == BAD
    assert scan(b=rows(b=2, d=32)) == BAD                      # S differs
    assert scan(c=rows(b=1, d=16)) == BAD                      # batch differs
    assert scan(b=rows(b=2, d=16, dtype=B.LA_F32)) == BAD
    assert scan(S=24, b=rows(b=2, d=24), c=rows(b=2, d=24)) == UNS
    assert scan(S=128, b=rows(b=2, d=128), c=rows(b=2, d=128)) == UNS
    assert scan(skip=0x30004) == BAD and scan(bias=0x30004) == BAD
    assert scan(sin=0x30004) == BAD and scan(sout=0x30004) == BAD and scan(lens=0x30001) == BAD
    assert scan(sin=0x30000, sout=0x30000) == BAD
    assert scan(out=rows(b=2, sn=32, sb=256)) == BAD
    assert scan(x=rows(b=2, sn=70)) == BAD
    z = rows(b=0)
    assert scan(x=z, dt=z, out=z, b=rows(b=0, d=16), c=rows(b=0, d=16)) == OK


def test_step_refusals():
    f = la.load().la_selective_step
    one, bc = rows(b=2, n=1), rows(b=2, n=1, d=16)

    def step(state=0x30000, x=one, S=16):
        return f(state, ref(x), ref(x), 0x20000, S, ref(bc), ref(bc), None, None, None, 1, ref(x),
                 None)
    assert step(state=None) == BAD and step(state=0x30004) == BAD
    assert step(x=rows(b=2, n=2)) == BAD
    assert step(S=8) == BAD                                    # b, c have 16


def test_python_checks():
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        la.causal_conv(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        la.linear(x, torch.zeros(8, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        la.selective_step(None, x[:, 0], x[:, 0], w, x[:, 0], x[:, 0])
    with pytest.raises(ValueError, match="activation"):
        la.linear(x, w, activation="tanh")
    with pytest.raises(ValueError, match="dtype"):
        la.linear(x.half(), w.half())
    with pytest.raises(TypeError):
        la.linear([1.0], w)
    with pytest.raises(TypeError):
        la.causal_conv(None, w)


def test_public_names():
    for name in ("linear", "causal_conv", "causal_conv_step", "selective_scan", "selective_step"):
        assert name in la.__all__ and callable(getattr(la, name))
