"""Properties of MX calls that a bound on the error alone does not show: a
token's bits whatever else is in its batch, the norm in place on rows that
start anywhere, and every stage of the feed-forward example on its own.

Tolerances: equal bits for the first two.  The example's products are held to
test_gpu_mx's bound for sums of exact products and their rounding to bfloat16;
its norm and SwiGLU to the roundings derived there."""
import importlib.util
import os

import numpy as np
import pytest

import mx_reference as ref
from test_gpu_mx import TYPES, _assert_padding, _assert_product, _assert_rounds, _dev, _q, _random_mx, _rng, _torch

pytestmark = pytest.mark.gpu


def _rows_of(mx, rows):
    """An MX tensor of the given rows of another."""
    q, torch = _q(), _torch()
    byte = ref.untile(mx.scales.cpu().numpy(), mx.rows)
    at = torch.as_tensor(rows).cuda()
    return q.MxTensor(mx.codes[at].contiguous(), torch.from_numpy(ref.tile(byte[rows])).cuda(), mx.K, mx.bits)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,N", [(5, 4096, 300), (16, 2560, 130), (60, 4096, 600), (200, 8192, 300), (300, 1152, 4100),
                                   (420, 2048, 4900), (700, 640, 3400)])
def test_the_bits_of_a_token_whatever_its_batch(T, K, N, bits):
    q, torch = _q(), _torch()
    g = _rng(71, T, bits)
    x, _ = _random_mx(g, T, K, bits)
    other, _ = _random_mx(g, T, K, bits)
    w, _ = _random_mx(g, N, K, 4)
    y = q.mx_matmul(x, w)
    order = g.permutation(T)
    moved = q.mx_matmul(_rows_of(x, order), w)          # every token at another place
    assert torch.equal(moved, y[torch.from_numpy(order).cuda()])
    keep = np.sort(g.choice(T, max(1, T // 3), replace=False))
    codes, byte = other.codes.clone(), ref.untile(other.scales.cpu().numpy(), T).copy()
    at = torch.from_numpy(keep).cuda()
    codes[at] = x.codes[at]
    byte[keep] = ref.untile(x.scales.cpu().numpy(), T)[keep]
    among = q.mx_matmul(q.MxTensor(codes, torch.from_numpy(ref.tile(byte)).cuda(), K, bits), w)   # among others
    assert torch.equal(among[at], y[at])


@pytest.mark.parametrize("which", ["x", "residual", "both"])
@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows,K", [(2000, 1001), (700, 4095), (300, 4096), (400, 40001), (2500, 17), (300, 9001)])
def test_rmsnorm_in_place_on_rows_that_start_anywhere(rows, K, name, which):
    # Neighbouring rows lie side by side, so that loads of whole granules reach
    # into rows that other CTAs are writing.
    q, torch = _q(), _torch()
    gen = torch.Generator(device="cuda").manual_seed(rows + K)
    x, r, w = (torch.randn(n, K, generator=gen, device="cuda").to(getattr(torch, name)) for n in (rows, rows, 1))
    if which == "both":
        r = x
    want, wh = q.mx_rmsnorm(x, w[0], residual=r)
    for _ in range(3):
        x1 = x.clone()
        r1 = x1 if which == "both" else r.clone()
        target = r1 if which == "residual" else x1
        got, h = q.mx_rmsnorm(x1, w[0], residual=r1, h_out=target)
        assert h is target and torch.equal(h, wh)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
        if which != "both":
            assert torch.equal(x1 if which == "residual" else r1, x if which == "residual" else r)


@pytest.mark.parametrize("tokens", [1, 30, 260])
def test_every_stage_of_the_feed_forward_example(tokens, monkeypatch):
    q, torch = _q(), _torch()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "llama_ffn_mx.py")
    spec = importlib.util.spec_from_file_location("llama_ffn_mx", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    seen = []

    class Calls:
        def __getattr__(self, name):
            def call(*a, **kw):
                out = getattr(q, name)(*a, **kw)
                seen.append((name, a, out))
                return out
            return call

    monkeypatch.setattr(ex, "q4mm", Calls())
    dim, hidden = 768, 1100
    weights, x, residual = ex.make(dim, hidden, tokens, seed=tokens)
    block = ex.MxFeedForward(**weights)
    y, h = block(x, residual)
    assert [s[0] for s in seen] == ["mx_quantize", "mx_quantize", "mx_rmsnorm", "mx_matmul", "mx_swiglu", "mx_matmul"]

    def value(t):
        return (q.mx_dequantize(t) if isinstance(t, q.MxTensor) else t).double().cpu().numpy()

    for (_, (w,), mx), parts in zip(seen[:2], (("gate", "up"), ("down",))):
        assert torch.equal(w, torch.cat([weights[p] for p in parts]))
        codes, byte = ref.quantize(value(w), 4)
        assert np.array_equal(value(mx), ref.values(codes, byte, 4)[:, :mx.K])
    n = seen[2][2][0]
    v, _ = ref.rmsnorm(value(x), value(weights["norm"]), float(np.float32(block.eps)), value(residual))
    _assert_rounds(n, v, 3e-6 * np.abs(v))
    gu = seen[3][2]
    assert seen[3][1] == (n, block.gate_up) and gu.dtype == torch.bfloat16
    _assert_product(gu, value(n), value(block.gate_up), "bfloat16")
    a = seen[4][2]
    v = ref.swiglu(value(gu[:, :hidden]), value(gu[:, hidden:]))
    _assert_rounds(a, v, 1e-6 * np.abs(v))
    _assert_padding(a)
    assert seen[5][1] == (a, block.down) and seen[5][2] is y
    _assert_product(y, value(a), value(block.down), "bfloat16")
    assert torch.equal(h, x + residual)
