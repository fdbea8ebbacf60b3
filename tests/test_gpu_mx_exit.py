"""How the MX products leave an SM: the next kernel's CTAs take it over at
once, so nothing of the last one (a signal, a copy) may still be under way.
Kernels of both forms run back to back without a gap, and every result has
the bits of a call on its own."""
import pytest

from test_gpu_mx import _random_mx, _rng

pytestmark = pytest.mark.gpu

# CTA pairs with one and two blocks of K a stage, one and several tiles to a pair; single CTAs, split and whole.
SIZES = [(700, 640, 3400), (100, 384, 50000), (16, 2560, 130), (420, 2048, 4900), (1, 4096, 300), (20, 300, 20000)]


def _torch():
    import torch
    return torch


def _q():
    import quantized_matmul_q4_gb300 as q
    return q


def _products(bits):
    q = _q()
    ops = []
    for T, K, N in SIZES:
        g = _rng(51, T, K, N)
        ops.append((_random_mx(g, T, K, bits)[0], _random_mx(g, N, K, 4)[0]))
    want = []
    for x, w in ops:
        want.append(q.mx_matmul(x, w))
        _torch().cuda.synchronize()
    return ops, want


@pytest.mark.parametrize("bits", [4, 8])
def test_products_back_to_back(bits):
    q, torch = _q(), _torch()
    ops, want = _products(bits)
    outs = [torch.empty_like(y) for y in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            for (x, w), y in zip(ops, outs):
                q.mx_matmul(x, w, out=y)
    for _ in range(25):
        for y in outs:
            y.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(y, t) for y, t in zip(outs, want))
    q.device_status()

