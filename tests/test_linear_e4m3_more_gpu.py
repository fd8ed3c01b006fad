"""Products of 8-bit operands on the GPU: scales at the ends of fp32's range, and every
kernel that the sizes lead to."""
import pytest
import torch

import causal_kernelized_linear_gb300 as la
from test_delta_block_gpu import BF16, DEV, E4M3, U, _f, _gen, _linear8, _linear8_close

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


# m, k, n, and the kernel on 152 SMs: split K, rings that wrap, tiles that follow one another
KERNELS = [
    (16, 4096, 520, "few16"), (64, 4096, 520, "few32"), (200, 4096, 2048, "few64"), (100, 4112, 4096, "few64"),
    (3000, 4096, 520, "few128"), (5000, 1104, 264, "few128"), (2013, 1184, 2392, "pair128"), (12277, 2800, 264, "pair128"),
    (4100, 2064, 2568, "pair256"), (2300, 4096, 1032, "pair256")]


@pytest.mark.parametrize("m,k,n,kernel", KERNELS)
def test_every_kernel(m, k, n, kernel):
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert la.selftest_linear_kernel(E4M3, m, n, k) == kernel
    args = _linear8(m, k, n, m + k + n)
    x, xs, w, ws, bias, residual = args
    y = la.linear_e4m3(x, xs, w, ws, bias=bias, residual=residual)
    _linear8_close(y, *args)
    assert torch.equal(y, la.linear_e4m3(x, xs, w, ws, bias=bias, residual=residual))
    none = la.linear_e4m3(x, xs, w, ws, activation="gelu")
    _linear8_close(none, x, xs, w, ws, None, None, act="gelu")
    # rows and columns of a larger output keep to themselves
    big = torch.full((m + 2, n + 16), 7.0, device=DEV, dtype=BF16)
    out = la.linear_e4m3(x, xs, w, ws, activation="gelu", out=big[1:-1, 8:-8])
    assert torch.equal(out, none)
    for edge in (big[0], big[-1], big[:, :8], big[:, -8:]):
        assert (edge == 7).all()
