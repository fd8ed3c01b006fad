"""Which kernel a product or a step runs, from the sizes alone (no GPU needed)."""
import math
import random

import pytest
import torch

import causal_kernelized_linear_gb300 as la

SMS = 152


@pytest.fixture(scope="module", autouse=True)
def lib():
    la.build()


def test_every_kernel_of_linear_is_reached():
    rng = random.Random(1)
    seen = set()
    for _ in range(20000):
        m, k, n = (int(math.exp(rng.uniform(math.log(lo), math.log(hi))))
                   for lo, hi in ((1, 16384), (64, 4096), (64, 8192)))
        for dtype in (torch.bfloat16, torch.float32):
            seen.add((dtype, la.selftest_linear_kernel(dtype, m, max(8, n // 8 * 8), max(8, k // 8 * 8), SMS)))
    assert seen == {(torch.bfloat16, n) for n in ("few16", "few32", "few64", "few128", "pair128", "pair256")} \
        | {(torch.float32, n) for n in ("rows2", "rows8", "tile8x1", "tile8x2", "tile8x4",
                                        "tile4x1", "tile4x2", "tile4x4")}


def test_kernel_of_the_step():
    assert la.selftest_step_kernel(1, 4096, 16, SMS) == "step1"
    assert la.selftest_step_kernel(256, 4096, 16, SMS) == "step4"
    assert la.selftest_step_kernel(3, 1 << 20, 64, SMS) == "step1"


def test_out_of_range():
    for bad in ((0, 8, 8), (8, 0, 8), (8, 8, 0), ((1 << 30) + 1, 8, 8)):
        with pytest.raises(ValueError):
            la.selftest_linear_kernel(torch.float32, *bad, SMS)
    with pytest.raises(ValueError):
        la.selftest_linear_kernel(torch.float32, 8, 8, 8, 0)
    for bad in ((0, 8, 8), (8, 0, 8), (8, 8, 24), ((1 << 24) + 1, 8, 8)):
        with pytest.raises(ValueError):
            la.selftest_step_kernel(*bad, SMS)
