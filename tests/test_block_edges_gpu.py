"""State-space block operators on the GPU: order with the kernels before them,
accuracy where a value is small, aliases, gradients and the sizes at which
another kernel takes over."""
import ctypes
import math

import pytest
import torch

import causal_kernelized_linear_gb300 as la

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, device=DEV, generator=g) * scale).to(dtype)


# ------------------------------------------------------------------ order with the kernel before

def _edges(f):
    """(edges, programmatic ones among them) of the graph that f's calls record."""
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        f()
    get = la.load().cudaGraphGetEdges            # from the CUDA runtime that the library is linked to
    get.argtypes = [ctypes.c_void_p] * 5
    n = ctypes.c_size_t()
    raw = graph.raw_cuda_graph()
    assert get(raw, None, None, None, ctypes.byref(n)) == 0
    ends = [(ctypes.c_void_p * max(1, n.value))() for _ in range(2)]
    data = (ctypes.c_uint8 * (8 * max(1, n.value)))()   # from_port, to_port, type, reserved
    assert get(raw, ends[0], ends[1], data, ctypes.byref(n)) == 0
    return n.value, sum(data[8 * i + 2] == 1 for i in range(n.value))


def test_scan_does_not_start_in_its_predecessors_tail():
    g = _gen(1)
    x, dt, gate = (_randn(g, 1, 100, 64) for _ in range(3))
    b, c = _randn(g, 1, 100, 16), _randn(g, 1, 100, 16)
    a = -torch.rand(64, 16, device=DEV, generator=g)
    w, cw = _randn(g, 64, 64), _randn(g, 64, 4)
    out = torch.empty_like(x)

    def conv_scan():
        la.selective_scan(la.causal_conv(x, cw), dt, a, b, c, gate=gate, out=out)

    def linear_scan():
        la.selective_scan(x, la.linear(x, w), a, b, c, gate=gate, out=out)

    def conv_linear():
        la.linear(la.causal_conv(x, cw), w, out=out)
    assert _edges(conv_linear) == (1, 1)         # the others still overlap
    assert _edges(conv_scan) == (1, 0)
    assert _edges(linear_scan) == (1, 0)


def test_single_round_of_fp32_tiles_does_not_start_in_its_predecessors_tail():
    g = _gen(2)
    f32 = torch.float32
    x = _randn(g, 400, 1024, dtype=f32)
    w = _randn(g, 512, 1024, dtype=f32, scale=1 / 32)
    cw = _randn(g, 1024, 4, dtype=f32)

    def conv_linear():
        la.linear(la.causal_conv(x[None], cw), w)
    assert _edges(conv_linear) == (1, 0)
