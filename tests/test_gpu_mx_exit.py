"""How the MX products leave an SM: the next kernel's CTAs take it over at
once, so nothing of the last one (a signal, a copy) may still be under way.
Kernels of both forms run back to back without a gap, also after a wait that
ran out, and every result has the bits of a call on its own."""
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



@pytest.mark.parametrize("stage", [0, 2])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,N", [(300, 4096, 5000), (1200, 2048, 2050), (192, 4224, 9000)])
def test_products_right_behind_a_wait_that_runs_out(T, K, N, bits, stage):
    q, torch = _q(), _torch()
    g = _rng(52, T, bits)
    x, _ = _random_mx(g, T, K, bits)
    w, _ = _random_mx(g, N, K, 4)
    ops, want = _products(bits)
    torch.cuda.synchronize()
    q.device_status()
    q.arm_wait_failure(stage, 2_000_000)
    q.mx_matmul(x, w)
    got = [q.mx_matmul(*o) for o in ops]
    torch.cuda.synchronize()
    with pytest.raises(q.Q4mmError) as e:
        q.device_status()
    assert e.value.code == -5
    assert all(torch.equal(y, t) for y, t in zip(got, want))
