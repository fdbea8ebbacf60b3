"""Attention over caches whose lengths and values lie at the ends of what the types hold.

Tolerances as derived in test_gpu_attention.
"""
import numpy as np
import pytest

import attention_reference as ref
import test_gpu_attention as base
import test_gpu_attention_batches as batches
from test_gpu_attention import KERNELS, Case, kernel  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _q():
    import quantized_matmul_q4_gb300 as q
    return q


def test_lengths_up_to_the_last_position():
    """A sequence of 2^31 - 256 tokens, whose table repeats one page of 2^24, gives what that page gives; a longer one is
    reported, as is one that is longer than its table.  The keys are shared by 15 clusters of 8 CTAs of 8 warps at least, each
    of which adds 2^31 / 960 / 16 < 2^18 times and drops at most 2^-23 of the sum each time."""
    q, torch = _q(), _torch()
    page = 2 ** 24
    cache = q.mx_cache(1, 1, 32, page=page, bits=4)
    g = torch.Generator(device="cuda").manual_seed(1)
    cache.k_codes.random_(0, 256, generator=g), cache.v_codes.fill_(0x22)       # values of v: 1
    cache.k_scales.fill_(125), cache.v_scales.fill_(127)
    x = torch.randn(1, 8, 32, generator=g, device="cuda")
    starts, table = base._i32([0, 1]), torch.zeros(1, 129, dtype=torch.int32, device="cuda")
    q.device_status()
    for dtype in (torch.float32, torch.bfloat16):
        y = q.mx_attention(x.to(dtype), cache, starts, base._i32([2 ** 31 - 256]), table)
        q.device_status()
        assert float((y.float() - 1).abs().max()) <= 2.0 ** -5 + base._half(str(dtype)[6:])
    for n, width in ((2 ** 31 - 1, 129), (2 ** 31 - 200, 129), (2 ** 24 + 1, 1)):
        q.mx_attention(x, cache, starts, base._i32([n]), table[:, :width].contiguous())
        with pytest.raises(q.Q4mmError) as e:
            q.device_status()
        assert e.value.code == -7


# Powers of two by which the values of neighbouring groups of tokens differ, in turn; None: all zeros.
POWERS = {"zeros": [None, 0, None], "zeros beside 2^50": [None, 50], "2^50 beside zeros": [50, None, None], "2^100, then zeros": [100, None],
          "far apart": [0, -60, 60, 100, None, -100], "up": [-100, 0, 100], "down": [100, 0, -100], "a step": [0, 0, 45], "tiny": [-112],
          "tiny, and zeros": [None, -112], "huge": [112, 112, 90]}


def _spread(scales, codes, powers, run):
    """Scale bytes [..., places, 4] and codes of v, in runs of `run` tokens, moved by the powers in turn."""
    torch = _torch()
    at = torch.arange(scales[..., 0].numel(), device=scales.device).view(scales.shape[:-1]) // run % len(powers)
    for i, p in enumerate(powers):
        mine = (at == i)[..., None]
        if p is None:
            scales.masked_fill_(mine, 0), codes.masked_fill_(mine, 0)
        else:
            scales.copy_(torch.where(mine, (scales.int() + p).clamp(0, 246), scales.int()).to(torch.uint8))


@KERNELS
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("run", [1, 16, 64])
@pytest.mark.parametrize("news,lengths,bits", [([1], [900], 8), ([1], [30000], 4), ([150], [700], 8), ([3, 20], [60, 333], 4)])
@pytest.mark.parametrize("powers", POWERS)
def test_values_of_any_powers(powers, news, lengths, bits, run, dtype):
    """Groups of tokens whose values differ by any powers of two, zeros among them: each counts in the sum of probabilities
    by its scores alone."""
    q = _q()
    b = batches.Batch(news, lengths, 2, 64, 64, bits, seed=run)
    _spread(b.cache.v_scales, b.cache.v_codes, POWERS[powers], run)
    x = b.queries(4, dtype, size=1.0)
    y = q.mx_attention(x, b.cache, *b.batch)
    q.device_status()
    assert bool(_torch().isfinite(y).all())
    b.check(x, y)


@KERNELS
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("high,low", [(60, -60), (100, -20), (20, -110), (0, -110)])
def test_small_values_of_large_probability(high, low, dtype):
    """Keys of tiny values whose probability makes them as large a part of the output as the huge values of keys of
    little probability, and far larger scores of keys without values."""
    q, torch = _q(), _torch()
    for n, m in ((1, 600), (140, 600)):
        c = Case(17, [n], [m], 1, 64, 16, 8).fill(size=0.01)
        gap = (high - low) * np.log(2)
        for p in range(m):
            pg, at, kind = c.table[0, p // 16], p % 16, p // 16 % 3
            s = c.cache["v_scales"][pg, 0, at]
            s[:2] = np.clip(s[:2].astype(int) + 6 + (high, low, 0)[kind], 0, 246)
            if kind == 2:
                c.cache["v_codes"][pg, 0, at], s[:] = 0, 0
            # k's first value alone makes the score: 0 for huge values, gap for tiny ones, a little less for none
            codes, byte = ref.head_codes(np.concatenate([[(0, 16, 15)[kind]], np.zeros(63)]), 8)
            c.cache["k_codes"][pg, 0, at], c.cache["k_scales"][pg, 0, at] = codes, byte
        x = np.zeros((n, 2, 64))
        x[..., 0] = gap / 16 * c.rng.uniform(0.9, 1.1, (n, 2))
        x, xv = base._dev(x, dtype)
        y = q.mx_attention(x, c.device_cache(), *c.device_batch(), scale=1.0)
        base._check(c, x, y, xv, dtype, scale=1.0)
