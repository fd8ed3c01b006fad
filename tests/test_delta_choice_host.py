"""Which kernel a product of 8-bit operands runs, and that every one has a test (no GPU needed)."""
import math
import random

import pytest
import torch

import causal_kernelized_linear_gb300 as la
from test_linear_e4m3_more_gpu import KERNELS

SMS, E4M3 = 152, torch.float8_e4m3fn
NAMES = {"few16", "few32", "few64", "few128", "pair128", "pair256"}


@pytest.fixture(scope="module", autouse=True)
def lib():
    la.build()


def test_every_kernel_has_a_tested_shape():
    for m, k, n, kernel in KERNELS:
        assert la.selftest_linear_kernel(E4M3, m, n, k, SMS) == kernel, (m, k, n)
    assert {kernel for *_, kernel in KERNELS} == NAMES


def test_every_kernel_is_reached():
    rng = random.Random(1)
    seen = set()
    for _ in range(20000):
        m, k, n = (int(math.exp(rng.uniform(math.log(lo), math.log(hi))))
                   for lo, hi in ((1, 16384), (64, 4096), (64, 8192)))
        seen.add(la.selftest_linear_kernel(E4M3, m, max(8, n // 8 * 8), max(16, k // 16 * 16), SMS))
    assert seen == NAMES


def test_out_of_range():
    for bad in ((0, 8, 16), (8, 0, 16), (8, 8, 0), ((1 << 30) + 1, 8, 16)):
        with pytest.raises(ValueError):
            la.selftest_linear_kernel(E4M3, *bad, SMS)
