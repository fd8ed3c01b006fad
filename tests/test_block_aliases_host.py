"""Outputs of the state-space block's operators that lie on their inputs: refused
before anything is queued (no GPU needed).

Every call here has to be refused: the addresses are not memory.  What has to be
let through is called with real memory by the GPU tests."""
import itertools
import random

import pytest

import causal_kernelized_linear_gb300 as la
from causal_kernelized_linear_gb300 import _binding as B
from test_block_host import BAD, conv, lib, lin, ref, rows, scan  # noqa: F401


def test_linear_output_over_input():
    P = 0x100000
    assert lin(x=rows(n=8, d=64, ptr=P), w=rows(n=64, d=64), out=rows(n=8, d=64, ptr=P)) == BAD
    assert lin(x=rows(n=8, d=64, ptr=P), out=rows(n=8, d=32, ptr=P + 1008)) == BAD   # its last bytes
    assert lin(x=rows(n=8, d=64, ptr=0x90000), w=rows(n=32, d=64, ptr=P), out=rows(n=8, d=32, ptr=P + 64)) == BAD
    # rows of one buffer, 256 apart: columns 0 to 63 read, 56 to 87 written
    assert lin(x=rows(n=8, d=64, ptr=P, sn=256), out=rows(n=8, d=32, ptr=P + 112, sn=256)) == BAD
    # the output a few rows further on
    assert lin(x=rows(n=8, d=64, ptr=P, sn=256), out=rows(n=8, d=32, ptr=P + 7 * 512 + 96, sn=256)) == BAD
    # a residual that is not the same view
    out = rows(n=8, d=32, ptr=P)
    assert lin(out=out, res=rows(n=8, d=32, ptr=P + 16)) == BAD
    assert lin(bias=P + 16, out=rows(n=8, d=32, ptr=P)) == BAD


def test_conv_output_over_input():
    P = 0x100000
    x = rows(b=2, ptr=P)
    assert conv(x=x, out=x) == BAD
    assert conv(x=x, out=rows(b=2, ptr=P + 1920)) == BAD
    assert conv(x=rows(b=2, ptr=P, sn=128), out=rows(b=2, ptr=P + 96, sn=128)) == BAD
    assert conv(out=rows(b=2, ptr=P), sin=P + 256) == BAD
    assert conv(out=rows(b=2, ptr=P), sout=P + 256) == BAD
    assert conv(x=x, out=rows(b=2, ptr=0x900000), sout=P) == BAD
    assert conv(out=rows(b=2, ptr=P), w=P + 512) == BAD
    assert conv(out=rows(b=2, ptr=P), lens=P + 512) == BAD
    # token-major memory: batch entries 64 apart, tokens 128
    t = rows(b=2, ptr=P, sb=64, sn=128)
    assert conv(x=t, out=rows(b=2, ptr=P + 16, sb=64, sn=128)) == BAD
    f, one = la.load().la_causal_conv_step, rows(b=2, n=1, ptr=P, sb=128)
    assert f(0x300000, ref(one), 0x20000, 4, None, 2, ref(rows(b=2, n=1, ptr=P + 64, sb=128)), None) == BAD
    assert f(P + 64, ref(one), 0x20000, 4, None, 2, ref(rows(b=2, n=1, ptr=0x900000)), None) == BAD
    assert f(P, ref(rows(b=2, n=1)), 0x20000, 4, None, 2, ref(one), None) == BAD


def test_scan_output_over_input():
    P = 0x100000
    out = rows(b=2, ptr=P)
    for k in ("x", "dt", "gate"):
        assert scan(out=out, **{k: rows(b=2, ptr=P + 16)}) == BAD      # another view of the same memory
    assert scan(out=out, b=rows(b=2, d=16, ptr=P)) == BAD
    assert scan(out=out, c=rows(b=2, d=16, ptr=P + 1024)) == BAD
    # b and c shared by the batch and the tokens: strides of zero
    assert scan(out=out, c=rows(b=2, d=16, ptr=P + 1024, sb=0, sn=0)) == BAD
    for k in ("a", "skip", "bias", "sin", "sout", "lens"):
        assert scan(out=out, **{k: P + 1024}) == BAD, k
    assert scan(sout=0x10000 - 0x100) == BAD                            # over x, dt, b and c
    assert scan(sout=P, a=P + 64) == BAD
    f, one, bc = la.load().la_selective_step, rows(b=2, n=1), rows(b=2, n=1, d=16, ptr=0x200000)

    def step(state=0x300000, x=one, out=one):
        return f(state, ref(x), ref(x), 0x20000, 16, ref(bc), ref(bc), None, None, None, 1, ref(out), None)
    assert step(out=rows(b=2, n=1, ptr=0x10000 + 64)) == BAD
    assert step(out=bc and rows(b=2, n=1, ptr=0x200000)) == BAD
    assert step(state=0x10000) == BAD and step(state=0x200000) == BAD and step(state=0x20000) == BAD


def test_all_small_views():
    """Views of a small buffer, every pair of the same strides: refused where the
    two sets of elements meet, counted one by one."""
    rng = random.Random(3)
    P, seen = 0x100000, 0
    for _ in range(4000):
        b, n, d = rng.choice([1, 2, 3]), rng.choice([1, 2, 5]), 8 * rng.choice([1, 2, 4])
        sn = rng.choice([d, d + 8, 2 * d, 4 * d])
        sb = rng.choice([n * sn, n * sn + 16])
        if rng.random() < 0.3:                # token-major
            sb, sn = sn, b * sn + rng.choice([0, 8])
        shift = 8 * rng.randrange(-2 * (b * n * 3), 2 * (b * n * 3))
        x = rows(b=b, n=n, d=d, ptr=P, sb=sb, sn=sn)
        out = rows(b=b, n=n, d=d, ptr=P + 2 * shift, sb=sb, sn=sn)
        at = [{i * sb + t * sn + c + s for i, t, c in itertools.product(range(b), range(n), range(d))}
              for s in (0, shift)]
        if not at[0] & at[1]:
            continue
        seen += 1
        far = dict(dt=rows(b=b, n=n, d=d, ptr=0x900000), b=rows(b=b, n=n, d=16, ptr=0xA00000),
                   c=rows(b=b, n=n, d=16, ptr=0xB00000))
        if shift:
            assert scan(x=x, out=out, **far) == BAD, (b, n, d, sb, sn, shift)
        assert conv(x=x, out=out, w=0xC00000) == BAD, (b, n, d, sb, sn, shift)
    assert seen > 500
