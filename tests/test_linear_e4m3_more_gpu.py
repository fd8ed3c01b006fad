"""Products of 8-bit operands on the GPU: scales at the ends of fp32's range, and every
kernel that the sizes lead to."""
import pytest
import torch

import causal_kernelized_linear_gb300 as la
from test_delta_block_gpu import BF16, DEV, E4M3, U, _f, _gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [5, 300])
@pytest.mark.parametrize("x_scale,w_scale", [(2.0 ** -126, 1e-6), (3e-38, 1e-5), (1e30, 2.0 ** -126), (2e-20, 3e-20)])
def test_small_scales(m, x_scale, w_scale):
    # the scales' own product is subnormal or 0, the result is not
    g = _gen(m)
    k, n = 2048, 264
    x = (torch.rand(m, k, device=DEV, generator=g) * 300 + 100).to(E4M3)
    w = (torch.rand(n, k, device=DEV, generator=g) * 300 + 100).to(E4M3)
    xs = (1 + torch.rand(m, device=DEV, generator=g)) * x_scale
    ws = (1 + torch.rand(n, device=DEV, generator=g)) * w_scale
    y = la.linear_e4m3(x, xs, w, ws)
    ref = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    assert ref.abs().min() > 1e-37 and ref.abs().max() < 1e38
    # the sum (all of its terms are positive), the two products, and the output's rounding
    tol = (U[BF16] + 2 * _f(k + 4) + 2.0 ** -22) * ref
    assert ((y.double() - ref).abs() <= tol).all(), ((y.double() - ref).abs() / ref).max()
